"""More of what the serving operators refuse or plan on the host (no GPU needed)."""
import ctypes

from test_chunk_refusals import L, _chunk  # noqa: F401 (L: the library, a fixture)


def test_calls_of_very_many_sequences_stay_on_the_form_without_limited_waits(L):  # noqa: F811
    """The tensor cores' form, which needs a workspace, walks the sequences while parts of it wait under a limit."""
    sizes = dict(n_tokens=1 << 20, max_new=1000, max_pages=4096, window=0, sinks=0)
    need = [L.wenc_chunk_attention_workspace(ctypes.byref(_chunk(n_seqs=n, **sizes))) for n in (4, 1 << 20, (1 << 20) + 1, 1 << 25)]
    assert need[0] > 0 and need[1] == need[0] and need[2:] == [0, 0]
