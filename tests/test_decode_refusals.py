"""What the decode-side entry points refuse, on the host (no GPU needed): bad sizes, pointers,
strides and types, before any device call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    from transformer_encoder_gb300 import lib
    from transformer_encoder_gb300.build import build
    build()
    return lib()


def _attn(**kw):
    from transformer_encoder_gb300.wenc import PrefixAttentionArgs
    a = PrefixAttentionArgs(dtype=1, n_seqs=4, q_len=1, n_heads=8, n_kv_heads=4, head_dim=64, q=256, out=256, q_stride=512,
                            out_stride=512, n_groups=2, max_group=2, k_prefix=256, v_prefix=256, k_group_stride=2560,
                            k_token_stride=256, v_group_stride=2560, v_token_stride=256, prefix_max=10, k_pages=256,
                            v_pages=256, k_page_stride=4096, v_page_stride=4096, n_pages=9, page_size=16, block_table=256,
                            block_table_stride=3, max_pages=3, lens=256, scale=0.125)
    for k, v in kw.items():
        assert hasattr(a, k)
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status,word", [
    (dict(dtype=2), 1, b"dtype"), (dict(head_dim=128), 2, b"head_dim"), (dict(n_seqs=0), 1, b"n_seqs"),
    (dict(q_len=0), 1, b"q_len"), (dict(n_heads=6), 1, b"multiple"), (dict(q=None), 1, b"NULL"),
    (dict(out=None), 1, b"NULL"), (dict(v_prefix=None), 1, b"together"), (dict(k_pages=None), 1, b"together"),
    (dict(k_prefix=None, v_prefix=None, k_pages=None, v_pages=None), 1, b"neither"),
    (dict(n_groups=0), 1, b"n_groups"), (dict(n_groups=3), 1, b"group_start"), (dict(max_group=5), 1, b"max_group"),
    (dict(prefix_max=0), 1, b"prefix_max"), (dict(prefix_max=(1 << 30) + 1), 2, b"prefix_max"),
    (dict(n_pages=0), 1, b"n_pages"), (dict(page_size=0), 1, b"page_size"), (dict(max_pages=0), 1, b"max_pages"),
    (dict(max_pages=1 << 27, block_table_stride=1 << 27), 2, b"2^30"), (dict(block_table=None), 1, b"block_table"),
    (dict(lens=None), 1, b"lens"), (dict(q_stride=504), 1, b"stride"), (dict(out_stride=511), 1, b"stride"),
    (dict(k_token_stride=128), 1, b"stride"), (dict(k_page_stride=2048), 1, b"stride"), (dict(q_stride=516), 1, b"16 bytes"),
    (dict(k_group_stride=-8), 1, b"stride"), (dict(block_table_stride=2), 1, b"block_table_stride"),
    (dict(q=264), 1, b"aligned"), (dict(v_pages=258), 1, b"aligned"), (dict(n_heads=8192, n_kv_heads=8192), 2, b"heads"),
    (dict(n_seqs=1 << 28, q_len=2, max_group=1 << 27), 2, b"tokens"),
    (dict(n_seqs=1 << 22, n_heads=4096, max_group=1 << 21, q_stride=1 << 20, out_stride=1 << 20), 2, b"rows"),
    (dict(k_page_stride=1 << 36), 2, b"2^36"),
])
def test_prefix_attention_refuses(L, kw, status, word):
    a = _attn(**kw)
    assert L.wenc_prefix_attention(ctypes.byref(a), None) == status
    assert word in L.wenc_last_error(), L.wenc_last_error()


def test_prefix_attention_workspace_is_sized_on_the_host(L):
    assert L.wenc_prefix_attention(None, None) == 1
    assert L.wenc_prefix_attention_workspace(None) == 0
    assert L.wenc_prefix_attention_workspace(ctypes.byref(_attn(head_dim=32))) == 0
    assert L.wenc_prefix_attention_workspace(ctypes.byref(_attn())) == 0  # 4 rows per key head: joined on chip
    many = dict(n_seqs=200, n_groups=1, max_group=200)
    both = L.wenc_prefix_attention_workspace(ctypes.byref(_attn(**many)))
    assert both >= 2 * 200 * 8 * (64 * 4 + 8)  # at least a share of the prefix and one of the own keys
    a = _attn(**many, workspace=256, workspace_bytes=both - 1)
    assert L.wenc_prefix_attention(ctypes.byref(a), None) in (1, 2)  # too small (or, first, no sm_103a device)


def test_the_binding_packs_the_structures_as_declared():
    from transformer_encoder_gb300 import wenc
    for cls, pack in ((wenc.PrefixAttentionArgs, wenc._PREFIX_PACK), (wenc.KvAppendArgs, wenc._APPEND_PACK)):
        values = [i + 1 for i in range(len(cls._fields_))]
        raw = pack.pack(*values)
        a = cls.from_buffer_copy(raw + bytes(ctypes.sizeof(cls) - len(raw)))
        assert [getattr(a, n) for n, _ in cls._fields_] == values


def _append(**kw):
    from transformer_encoder_gb300.wenc import KvAppendArgs
    a = KvAppendArgs(dtype=1, n_tokens=6, n_seqs=3, n_heads=8, n_kv_heads=4, head_dim=64, q=256, q_out=256, k=256, v=256,
                     q_stride=512, q_out_stride=512, k_stride=256, v_stride=256, k_pages=256, v_pages=256,
                     k_page_stride=4096, v_page_stride=4096, n_pages=9, page_size=16, block_table=256,
                     block_table_stride=3, max_pages=3, lens=256, inv_freq=256, rot_dim=64)
    for k, v in kw.items():
        assert hasattr(a, k)
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status,word", [
    (dict(k=None), 1, b"NULL"), (dict(v_pages=None), 1, b"NULL"), (dict(block_table=None), 1, b"NULL"),
    (dict(lens=None), 1, b"NULL"), (dict(q_out=None), 1, b"together"), (dict(dtype=3), 1, b"dtype"),
    (dict(head_dim=32), 2, b"head_dim"), (dict(n_seqs=0), 1, b"sizes"), (dict(n_tokens=-1), 1, b"sizes"),
    (dict(n_pages=0), 1, b"sizes"), (dict(page_size=0), 1, b"sizes"), (dict(n_heads=0), 1, b"n_heads"),
    (dict(n_kv_heads=5000), 2, b"heads"), (dict(max_pages=1 << 28, block_table_stride=1 << 28), 2, b"2^31"),
    (dict(n_tokens=7), 1, b"seq_start"), (dict(rot_dim=24), 2, b"rot_dim"), (dict(rot_dim=80), 2, b"rot_dim"),
    (dict(rot_dim=0), 2, b"rot_dim"), (dict(k_stride=248), 1, b"stride"), (dict(q_out_stride=256), 1, b"stride"),
    (dict(v_page_stride=4088), 1, b"page stride"), (dict(block_table_stride=1), 1, b"block_table_stride"),
    (dict(k=257), 1, b"aligned"), (dict(q_stride=516), 1, b"16 bytes"),
])
def test_kv_append_refuses(L, kw, status, word):
    a = _append(**kw)
    assert L.wenc_kv_append(ctypes.byref(a), None) == status
    assert word in L.wenc_last_error(), L.wenc_last_error()


def test_kv_append_without_tokens_needs_no_device(L):
    assert L.wenc_kv_append(None, None) == 1
    assert L.wenc_kv_append(ctypes.byref(_append(n_tokens=0)), None) == 0


def test_integer_product_refuses(L):
    p = ctypes.c_void_p(256)
    odd = ctypes.c_void_p(264)
    q = L.wenc_quantize_rows
    assert q(None, 0, p, p, 1, 64, None) == 1
    assert q(p, 2, p, p, 1, 64, None) == 1 and b"x_dtype" in L.wenc_last_error()
    assert q(p, 0, p, p, 0, 64, None) == 1
    assert q(p, 0, p, p, 1, 24, None) == 2
    assert q(p, 0, p, p, 1, 0, None) == 2
    assert q(odd, 0, p, p, 1, 64, None) == 1
    f = L.wenc_linear_i8
    big = 1 << 40
    assert f(None, p, p, p, p, None, p, 8, 128, 64, 0, p, big, None) == 1
    assert f(p, p, p, p, None, None, p, 8, 128, 64, 0, p, big, None) == 1
    assert f(p, p, p, p, p, None, p, 8, 128, 64, 3, p, big, None) == 1 and b"epilogue" in L.wenc_last_error()
    assert f(p, p, p, p, p, None, p, 8, 128, 64, 2, p, big, None) == 1 and b"resid" in L.wenc_last_error()
    assert f(p, p, p, p, p, None, p, 0, 128, 64, 0, p, big, None) == 1
    assert f(p, p, p, p, p, None, p, (1 << 28) + 1, 128, 64, 0, p, big, None) == 2
    assert f(p, p, p, p, p, None, p, 8, 100, 64, 0, p, big, None) == 2
    assert f(p, p, p, p, p, None, p, 8, 0, 64, 0, p, big, None) == 2
    assert f(p, p, p, p, p, None, p, 8, 128, 32, 0, p, big, None) == 2
    assert f(odd, p, p, p, p, None, p, 8, 128, 64, 0, p, big, None) == 1
    assert L.wenc_linear_i8_workspace(16, 51200, 6400) == 0  # few tokens: widened on the chip
    assert L.wenc_linear_i8_workspace(1 << 20, 5120, 1280) == 2 * 1280 * ((1 << 20) + 5120)
    assert L.wenc_linear_i8_workspace(0, 128, 64) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    from transformer_encoder_gb300 import kv_append, linear_i8, prefix_attention, quantize_rows
    q = torch.zeros(2, 1, 4, 64)
    k = torch.zeros(2, 8, 4, 64)
    with pytest.raises(TypeError):
        prefix_attention(q.half(), k, k)
    with pytest.raises(ValueError):
        prefix_attention(q[0], k, k)
    with pytest.raises(ValueError):
        prefix_attention(q)
    with pytest.raises(ValueError):
        prefix_attention(q, k)
    with pytest.raises(TypeError):
        quantize_rows(torch.zeros(2, 64))
    with pytest.raises(TypeError):
        linear_i8(torch.zeros(2, 64), None, None, None, None)
    with pytest.raises(ValueError):
        kv_append(q[0], k[0], k, k, None, None)
