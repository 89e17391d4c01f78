"""More of what the serving operators refuse or plan on the host (no GPU needed)."""
import ctypes

import pytest

import test_chunk_refusals
from test_chunk_refusals import L, _chunk, _extend, _i4, _release  # noqa: F401 (L: the library, a fixture)


def test_calls_of_very_many_sequences_stay_on_the_form_without_limited_waits(L):  # noqa: F811
    """The tensor cores' form, which needs a workspace, walks the sequences while parts of it wait under a limit."""
    sizes = dict(n_tokens=1 << 20, max_new=1000, max_pages=4096, window=0, sinks=0)
    need = [L.wenc_chunk_attention_workspace(ctypes.byref(_chunk(n_seqs=n, **sizes))) for n in (4, 1 << 20, (1 << 20) + 1, 1 << 25)]
    assert need[0] > 0 and need[1] == need[0] and need[2:] == [0, 0]


def test_the_steps_of_a_unit_on_the_tensor_cores(L):  # noqa: F811
    """Steps of 128 keys from the first visible one on, at any key (the other steps and alignments: test_chunk_refusals.py)."""
    test_chunk_refusals.test_the_steps_of_a_run_of_tokens(L, 128, 1)


# _chunk's 12 tokens of 8 heads: q and out 12288 bytes (bf16), pages 73728, table 48, lens 16, seq_start 20
CHUNK_APART = dict(q=1 << 20, out=2 << 20, k_pages=3 << 20, v_pages=4 << 20, block_table=5 << 20, lens=6 << 20, seq_start=7 << 20)


@pytest.mark.parametrize("kw", [
    dict(out=(3 << 20) + 73712), dict(k_pages=(2 << 20) + 12272), dict(out=(4 << 20) + 73712), dict(v_pages=(2 << 20) + 12272),
    dict(out=(5 << 20) + 32), dict(block_table=(2 << 20) + 12284), dict(lens=(2 << 20) - 12), dict(lens=(2 << 20) + 12284),
    dict(seq_start=(2 << 20) - 16), dict(seq_start=(2 << 20) + 12284), dict(k_page_stride=8192, out=(3 << 20) + 135168 + 3840),
])
def test_chunk_attention_refuses_an_output_over_its_inputs(L, kw):  # noqa: F811
    assert L.wenc_chunk_attention(ctypes.byref(_chunk(**{**CHUNK_APART, **kw})), None) == 1
    assert b"shares memory" in L.wenc_last_error(), L.wenc_last_error()


@pytest.mark.parametrize("kw", [
    dict(), dict(out=(3 << 20) + 73728), dict(out=(3 << 20) - 12288), dict(lens=(2 << 20) - 16), dict(seq_start=(2 << 20) + 12288),
    dict(block_table=(2 << 20) - 48), dict(seq_start=None, lens=(2 << 20) - 16),
])
def test_chunk_attention_takes_what_lies_side_by_side(L, kw):  # noqa: F811
    """(Without a GPU the call ends at the device, behind these checks.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    L.wenc_chunk_attention(ctypes.byref(_chunk(**{**CHUNK_APART, **kw})), None)
    assert b"shares" not in L.wenc_last_error() and b"apart" not in L.wenc_last_error(), L.wenc_last_error()


# M 4, N 256, K 256, group 64 of _i4: x 2048 bytes (bf16), w 32768, w_scale 2048, bias 1024, out 2048 (4096 with a residual)
APART = dict(x=1 << 20, w=2 << 20, w_scale=3 << 20, bias=4 << 20, out=5 << 20)


@pytest.mark.parametrize("kw", [
    dict(out=(2 << 20) + 32752), dict(w=(5 << 20) + 2032), dict(out=(3 << 20) + 2032), dict(bias=(5 << 20) + 2032), dict(out=(4 << 20) + 1008),
    dict(scale_dtype=0, out=(3 << 20) + 4080), dict(x=(5 << 20) + 2032), dict(x_dtype=0, x=(5 << 20) + 4080),
    # a residual that begins before the output or behind its begin
    dict(epilogue=2, resid=(5 << 20) - 4080), dict(epilogue=2, resid=(5 << 20) + 16), dict(epilogue=2, resid=(5 << 20) + 4080),
    # (20 tokens of float32: a workspace of 30720 bytes)
    dict(M=20, x_dtype=0, workspace=(1 << 20) + 20224), dict(M=20, x_dtype=0, workspace=(2 << 20) - 30464),
    dict(M=20, x_dtype=0, workspace=(3 << 20) - 30464), dict(M=20, x_dtype=0, workspace=4 << 20), dict(M=20, x_dtype=0, workspace=(5 << 20) + 20224),
    dict(M=20, x_dtype=0, epilogue=2, resid=6 << 20, workspace=(6 << 20) + 20224),
])
def test_linear_i4_refuses_what_overlaps(L, kw):  # noqa: F811
    assert _i4(L, **{**APART, "workspace_bytes": 1 << 20, **kw}) == 1
    assert b"apart" in L.wenc_last_error(), L.wenc_last_error()


@pytest.mark.parametrize("kw", [
    dict(), dict(epilogue=2, resid=5 << 20), dict(epilogue=2, resid=(5 << 20) + 4096), dict(epilogue=2, resid=(5 << 20) - 4096),
    dict(resid=(5 << 20) + 16), dict(out=(4 << 20) + 1024), dict(out=(1 << 20) - 2048), dict(M=16, x_dtype=0, workspace=1 << 20),
    dict(M=20, x_dtype=0, workspace=6 << 20), dict(M=20, workspace=1 << 20),
])
def test_linear_i4_takes_what_lies_side_by_side(L, kw):  # noqa: F811
    """(Without a GPU the call ends at the device, behind these checks.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    _i4(L, **{**APART, "workspace_bytes": 1 << 20, **kw})
    assert b"apart" not in L.wenc_last_error(), L.wenc_last_error()


# 3 sequences and 8 rows: lens_out 12 bytes at 8192, free_count_out 4 at 8448, seq_start 16 at 8704, positions 32 at 9216, slots 64 at
# 10240; the table 48 at 1024
@pytest.mark.parametrize("kw", [
    dict(free_pages=1024 + 44), dict(free_pages=1024 - 44), dict(lens=1024 + 44), dict(new_tokens=1024 - 8), dict(free_count=1024),
    dict(lens_out=8444), dict(free_count_out=8704 + 12), dict(seq_start=8192 + 8), dict(positions=10240 + 48), dict(slots=9216 - 48),
    dict(positions=8704), dict(slots=8192 - 48),
])
def test_kv_extend_refuses_what_it_writes_over_one_another(L, kw):  # noqa: F811
    assert L.wenc_kv_extend(ctypes.byref(_extend(**kw)), None) == 1
    assert b"apart" in L.wenc_last_error(), L.wenc_last_error()


@pytest.mark.parametrize("kw", [dict(lens_out=8444), dict(free_pages=8192 - 44), dict(free_pages=8192 + 8), dict(trimmed_out=8192 + 8),
                                dict(free_count_out=8704 + 8), dict(free_count_out=2048 + 44)])
def test_kv_release_refuses_what_it_writes_over_one_another(L, kw):  # noqa: F811
    assert L.wenc_kv_release(ctypes.byref(_release(**kw)), None) == 1
    assert b"apart" in L.wenc_last_error(), L.wenc_last_error()


@pytest.mark.parametrize("call,args", [("wenc_kv_extend", kw) for kw in (
    dict(), dict(free_pages=1024 + 48), dict(lens=1024 - 12), dict(lens_out=8448 - 12), dict(slots=9216 + 32))] + [("wenc_kv_release", kw) for kw in (
        dict(), dict(lens_out=8448 - 12), dict(free_pages=8192 - 48), dict(trimmed_out=8192 + 12))])
def test_page_plans_take_what_lies_side_by_side(L, call, args):  # noqa: F811
    """(Without a GPU the call ends at the device, behind these checks.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    getattr(L, call)(ctypes.byref((_extend if call == "wenc_kv_extend" else _release)(**args)), None)
    assert b"apart" not in L.wenc_last_error(), L.wenc_last_error()
