"""The binding of the decode-side calls without a GPU: tensors that say they are on device 0, and a library that records
what it is called with. What the binding accepts is what reaches the library, in the layout the library expects."""
import pytest


class _Lib:
    """Every function of the library: records its name and arguments and returns 0."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or 0


@pytest.fixture
def lib(monkeypatch):
    import torch
    from transformer_encoder_gb300 import wenc
    fake = _Lib()
    monkeypatch.setattr(wenc, "_torch", torch)
    monkeypatch.setattr(wenc, "_lib", fake)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    return fake


def _cache(hd=64, heads=4, n=3):
    import torch
    pages = torch.zeros(6, 8, heads, hd)
    table = torch.zeros(n, 2, dtype=torch.int32)
    return pages, table, torch.ones(n, dtype=torch.int32)


@pytest.mark.parametrize("hd", [32, 128])
def test_pages_of_another_head_width_are_refused(lib, hd):
    """Pages [n, size, heads, 128] would give a page stride that is merely larger than it has to be."""
    import torch
    from transformer_encoder_gb300 import kv_append, prefix_attention
    q, k = torch.zeros(3, 1, 4, 64), torch.zeros(3, 4, 64)
    prefix = torch.zeros(1, 5, 4, 64)
    pages, table, lens = _cache(hd)
    for kw in (dict(), dict(k_prefix=prefix, v_prefix=prefix)):
        with pytest.raises(ValueError, match="page_size, 4, 64"):
            prefix_attention(q, **kw, k_pages=pages, v_pages=pages, block_table=table, lens=lens)
    with pytest.raises(ValueError, match="page_size, 4, 64"):
        kv_append(k, k, pages, pages, table, lens)
    assert not lib.calls
    pages = _cache()[0]
    prefix_attention(q, prefix, prefix, k_pages=pages, v_pages=pages, block_table=table, lens=lens)
    kv_append(k, k, pages, pages, table, lens)
    assert [c[0] for c in lib.calls] == ["wenc_prefix_attention", "wenc_kv_append"]


def test_a_workspace_of_fewer_bytes_than_elements_is_refused(lib):
    """One byte that is expanded counts 2^30 elements; the library would write behind it."""
    import torch
    from transformer_encoder_gb300 import linear_i8, prefix_attention
    from transformer_encoder_gb300.wenc import _PREFIX_PACK
    q, prefix = torch.zeros(200, 1, 4, 64), torch.zeros(1, 5, 4, 64)
    a, w, f = torch.zeros(64, 128, dtype=torch.int8), torch.zeros(128, 128, dtype=torch.int8), torch.zeros(128)
    wide = torch.empty(1, dtype=torch.uint8).expand(1 << 30)
    strided = torch.empty(4096, dtype=torch.uint8)[::2]
    for ws in (wide, strided):
        with pytest.raises(ValueError, match="workspace"):
            prefix_attention(q, prefix, prefix, workspace=ws)
        with pytest.raises(ValueError, match="workspace"):
            linear_i8(a, f[:64], w, f, f, workspace=ws)
    assert not lib.calls
    room = torch.empty(1024, dtype=torch.float32)
    prefix_attention(q, prefix, prefix, workspace=room)
    linear_i8(a, f[:64], w, f, f, workspace=room)
    (_, (packed, _)), (_, args) = lib.calls
    assert _PREFIX_PACK.unpack(packed)[-2:] == (room.data_ptr(), 4096)
    assert args[11:13] == (room.data_ptr(), 4096)


def test_an_empty_batch_gives_an_empty_output(lib):
    import torch
    from transformer_encoder_gb300 import EPI_BIAS_RESID_F32, kv_append, linear_i8, prefix_attention, quantize_rows
    pages, table, lens = _cache(n=0)
    prefix = torch.zeros(2, 5, 4, 64)
    for kw in (dict(k_prefix=prefix, v_prefix=prefix), dict(k_prefix=prefix[:0], v_prefix=prefix[:0]),
               dict(k_pages=pages, v_pages=pages, block_table=table, lens=lens)):
        assert prefix_attention(torch.zeros(0, 1, 4, 64), **kw).shape == (0, 1, 4, 64)
    assert prefix_attention(torch.zeros(2, 0, 4, 64), prefix, prefix).shape == (2, 0, 4, 64)
    with pytest.raises(ValueError, match="groups"):
        prefix_attention(torch.zeros(3, 1, 4, 64), prefix, prefix)
    q, scale = quantize_rows(torch.zeros(2, 0, 64))
    assert q.shape == (2, 0, 64) and q.dtype is torch.int8 and scale.shape == (2, 0)
    w, f = torch.zeros(128, 64, dtype=torch.int8), torch.zeros(128)
    assert linear_i8(q[0], scale[0], w, f, f).shape == (0, 128)
    assert linear_i8(q[0], scale[0], w, f, f, EPI_BIAS_RESID_F32, resid=torch.zeros(0, 128)).dtype is torch.float32
    k = torch.zeros(0, 4, 64)
    assert kv_append(k, k, pages, pages, table, lens, q=k).shape == (0, 4, 64)
    assert not lib.calls
