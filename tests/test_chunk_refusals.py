"""What the chunk attention, the page plans and the 4-bit product refuse, on the host (no GPU needed), and the index
arithmetic that their kernels share with the host, against plain definitions."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def L():
    from transformer_encoder_gb300 import lib
    from transformer_encoder_gb300.build import build
    build()
    return lib()


def _set(a, kw):
    for k, v in kw.items():
        assert hasattr(a, k)
        setattr(a, k, v)
    return a


def _chunk(**kw):
    from transformer_encoder_gb300.wenc import ChunkAttentionArgs
    return _set(ChunkAttentionArgs(dtype=1, n_tokens=12, n_seqs=4, max_new=5, n_heads=8, n_kv_heads=4, head_dim=64, q=256, out=256,
                                   q_stride=512, out_stride=512, k_pages=256, v_pages=256, k_page_stride=4096,
                                   v_page_stride=4096, n_pages=9, page_size=16, block_table=256, block_table_stride=3,
                                   max_pages=3, lens=256, seq_start=256, window=20, sinks=4, scale=0.125), kw)


@pytest.mark.parametrize("kw,status,word", [
    (dict(dtype=2), 1, b"dtype"), (dict(head_dim=128), 2, b"head_dim"), (dict(n_seqs=0), 1, b"positive"),
    (dict(n_tokens=-1), 1, b"positive"), (dict(n_heads=0), 1, b"positive"), (dict(n_heads=6), 1, b"multiple"),
    (dict(max_new=0), 1, b"max_new"), (dict(max_new=13), 1, b"max_new"), (dict(seq_start=None, n_tokens=13), 1, b"seq_start"),
    (dict(seq_start=None, max_new=2), 1, b"max_new"), (dict(n_heads=8192, n_kv_heads=8192), 2, b"heads"),
    (dict(window=-1), 1, b"window"), (dict(sinks=-1), 1, b"sinks"), (dict(window=0), 1, b"sinks"),
    (dict(max_pages=1 << 27, block_table_stride=1 << 27), 2, b"2^30"), (dict(n_tokens=1 << 28, q_stride=1 << 20), 2, b"rows"),
    (dict(scale=float("nan")), 1, b"scale"), (dict(scale=float("inf")), 1, b"scale"), (dict(q=None), 1, b"NULL"),
    (dict(v_pages=None), 1, b"NULL"), (dict(block_table=None), 1, b"NULL"), (dict(lens=None), 1, b"NULL"),
    (dict(q_stride=504), 1, b"stride"), (dict(out_stride=511), 1, b"stride"), (dict(q_stride=516), 1, b"16 bytes"),
    (dict(k_page_stride=2048), 1, b"stride"), (dict(v_page_stride=4100), 1, b"16 bytes"), (dict(k_page_stride=1 << 36), 2, b"2^36"),
    (dict(block_table_stride=2), 1, b"block_table_stride"), (dict(q=264), 1, b"aligned"), (dict(out=258), 1, b"aligned"), (dict(), 1, b"apart"),
])
def test_chunk_attention_refuses(L, kw, status, word):
    assert L.wenc_chunk_attention(ctypes.byref(_chunk(**kw)), None) == status
    assert word in L.wenc_last_error(), L.wenc_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(scale=3e38), 1, b"scale"), (dict(scale=-2.4e38), 1, b"scale"),
    # out within q's rows: a head further on, before it, rows at another stride, the last row alone
    (dict(out=256 + 128), 1, b"apart"), (dict(q=256 + 128), 1, b"apart"), (dict(out=256 + 1024 * 3, out_stride=1024), 1, b"apart"),
    (dict(out=256 + 1024 * 11), 1, b"apart"), (dict(q_stride=1024, out_stride=1024, out=256 + 1008), 1, b"apart"),
])
def test_chunk_attention_refuses_what_overlaps(L, kw, status, word):
    assert L.wenc_chunk_attention(ctypes.byref(_chunk(**kw)), None) == status
    assert word in L.wenc_last_error(), L.wenc_last_error()


@pytest.mark.parametrize("kw", [
    dict(out=256 + 1024 * 12), dict(q=256 + 1024 * 12), dict(q_stride=1024, out_stride=1024, out=256 + 1024),
    dict(q_stride=1792, out_stride=1792, out=256 + 2048),
])
def test_chunk_attention_takes_rows_side_by_side(L, kw):
    """(Without a GPU the call ends at the device, behind every check of its arguments; a workspace is refused before it.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    L.wenc_chunk_attention(ctypes.byref(_chunk(**kw)), None)
    assert b"apart" not in L.wenc_last_error(), L.wenc_last_error()


def test_chunk_attention_without_tokens(L):
    assert L.wenc_chunk_attention(None, None) == 1
    assert L.wenc_chunk_attention_workspace(None) == 0
    assert L.wenc_chunk_attention_workspace(ctypes.byref(_chunk(n_tokens=0))) == 0
    assert L.wenc_chunk_attention(ctypes.byref(_chunk(n_tokens=0, max_new=0)), None) == 0


def _extend(**kw):
    from transformer_encoder_gb300.wenc import KvExtendArgs
    return _set(KvExtendArgs(n_seqs=3, n_rows=8, new_tokens=256, lens=512, block_table=1024, block_table_stride=4, max_pages=4,
                             page_size=16, free_pages=2048, n_free_pages=12, free_count=4096, lens_out=8192,
                             free_count_out=8448, seq_start=8704, positions=9216, slots=10240), kw)


@pytest.mark.parametrize("kw,status,word", [
    (dict(new_tokens=None), 1, b"NULL"), (dict(lens_out=None), 1, b"NULL"), (dict(free_count=None), 1, b"NULL"),
    (dict(positions=None), 1, b"NULL"), (dict(slots=None), 1, b"NULL"), (dict(n_seqs=-1), 1, b"positive"),
    (dict(page_size=0), 1, b"positive"), (dict(max_pages=0), 1, b"positive"), (dict(n_free_pages=0), 1, b"positive"),
    (dict(n_rows=-1), 1, b"positive"), (dict(n_seqs=65537), 2, b"sequences"), (dict(n_rows=0x7fffffff), 2, b"n_rows"),
    (dict(page_size=1 << 30), 2, b"2^31"), (dict(block_table_stride=3), 1, b"block_table_stride"),
    (dict(positions=9220), 1, b"aligned"), (dict(slots=10248), 1, b"aligned"), (dict(lens_out=512), 1, b"apart"),
    (dict(lens_out=520), 1, b"apart"), (dict(free_count_out=4096), 1, b"apart"), (dict(lens_out=260), 1, b"apart"),
    (dict(seq_start=500), 1, b"apart"), (dict(seq_start=244), 1, b"apart"),
])
def test_kv_extend_refuses(L, kw, status, word):
    assert L.wenc_kv_extend(ctypes.byref(_extend(**kw)), None) == status
    assert word in L.wenc_last_error(), L.wenc_last_error()


@pytest.mark.parametrize("kw", [dict(positions=512), dict(slots=496), dict(lens_out=2048 + 44), dict(positions=1024 + 32),
                                dict(free_count_out=2048), dict(seq_start=1024)])
def test_kv_extend_refuses_outputs_over_pages_and_tables(L, kw):
    assert L.wenc_kv_extend(ctypes.byref(_extend(**kw)), None) == 1
    assert b"apart" in L.wenc_last_error(), L.wenc_last_error()


def _release(**kw):
    from transformer_encoder_gb300.wenc import KvReleaseArgs
    return _set(KvReleaseArgs(n_seqs=3, lens=512, finished=256, block_table=1024, block_table_stride=4, max_pages=4, page_size=16,
                              window=20, sinks=4, trimmed=1536, free_pages=2048, n_free_pages=12, free_count=4096,
                              lens_out=8192, free_count_out=8448, trimmed_out=8704), kw)


@pytest.mark.parametrize("kw,status,word", [
    (dict(lens=None), 1, b"NULL"), (dict(block_table=None), 1, b"NULL"), (dict(free_count_out=None), 1, b"NULL"),
    (dict(finished=None, window=0, trimmed=None, trimmed_out=None), 1, b"neither"), (dict(trimmed=None), 1, b"trimmed"),
    (dict(trimmed=None, trimmed_out=None), 1, b"trimmed"), (dict(window=0), 1, b"trimmed"), (dict(window=-1), 1, b"trimmed"),
    (dict(sinks=-1), 1, b"sinks"), (dict(n_seqs=65537), 2, b"sequences"), (dict(n_free_pages=0), 1, b"positive"),
    (dict(page_size=1 << 30), 2, b"2^31"), (dict(block_table_stride=3), 1, b"block_table_stride"),
    (dict(lens_out=516), 1, b"apart"), (dict(trimmed_out=1536), 1, b"apart"), (dict(free_count_out=4096), 1, b"apart"),
    (dict(lens_out=1540), 1, b"apart"),
])
def test_kv_release_refuses(L, kw, status, word):
    assert L.wenc_kv_release(ctypes.byref(_release(**kw)), None) == status
    assert word in L.wenc_last_error(), L.wenc_last_error()


@pytest.mark.parametrize("kw", [dict(lens_out=256), dict(free_pages=1024), dict(free_pages=480), dict(trimmed_out=1064),
                                dict(free_count_out=256)])
def test_kv_release_refuses_outputs_over_marks_and_tables(L, kw):
    assert L.wenc_kv_release(ctypes.byref(_release(**kw)), None) == 1
    assert b"apart" in L.wenc_last_error(), L.wenc_last_error()


def _i4(L, **kw):
    d = dict(x=256, x_dtype=1, w=256, w_scale=256, scale_dtype=1, bias=256, resid=None, out=256, M=4, N=256, K=256, group=64,
             epilogue=0, workspace=None, workspace_bytes=0, stream=None)
    assert set(kw) <= set(d)
    return L.wenc_linear_i4(*{**d, **kw}.values())


@pytest.mark.parametrize("kw,status,word", [
    (dict(x=None), 1, b"NULL"), (dict(bias=None), 1, b"NULL"), (dict(x_dtype=2), 1, b"dtype"), (dict(scale_dtype=-1), 1, b"dtype"),
    (dict(epilogue=3), 1, b"epilogue"), (dict(epilogue=2), 1, b"resid"), (dict(M=0), 1, b"M"), (dict(M=(1 << 28) + 1), 2, b"2^28"),
    (dict(N=64), 2, b"128"), (dict(N=192), 2, b"128"), (dict(K=64), 2, b"128"), (dict(K=192), 2, b"128"),
    (dict(group=16), 2, b"group"), (dict(group=256), 2, b"group"), (dict(group=96), 2, b"group"), (dict(x=264), 1, b"aligned"),
    (dict(w=260), 1, b"aligned"), (dict(w_scale=258), 1, b"aligned"), (dict(out=264), 1, b"aligned"),
])
def test_linear_i4_refuses(L, kw, status, word):
    assert _i4(L, **kw) == status
    assert word in L.wenc_last_error(), L.wenc_last_error()


@pytest.mark.parametrize("kw", [dict(), dict(out=256 + 2032), dict(x=256 + 2032), dict(epilogue=2, resid=65536, x=256 + 4080),
                                dict(x_dtype=0, out=256 + 4080)])
def test_linear_i4_refuses_an_output_over_its_input(L, kw):
    assert _i4(L, **kw) == 1
    assert b"apart" in L.wenc_last_error(), L.wenc_last_error()


def test_the_binding_packs_the_structures_as_declared():
    from transformer_encoder_gb300 import wenc
    for cls, pack in ((wenc.ChunkAttentionArgs, wenc._CHUNK_PACK), (wenc.KvExtendArgs, wenc._EXTEND_PACK),
                      (wenc.KvReleaseArgs, wenc._RELEASE_PACK)):
        values = [i + 1 for i in range(len(cls._fields_))]
        a = cls.from_buffer_copy(pack.pack(*values))
        assert [getattr(a, n) for n, _ in cls._fields_] == values


@pytest.mark.parametrize("step,align", [(16, 16), (128, 8), (128, 16), (128, 128), (64, 1)])
def test_the_steps_of_a_run_of_tokens(L, step, align):
    """Every key that one of the tokens sees is in one step, and no other key is loaded."""
    r = np.random.default_rng(step + align)
    for _ in range(400):
        first = int(r.integers(-5, 700))
        last = first + int(r.choice([0, 0, 1, 5, 60, 200]))
        window, sinks = (int(r.choice([1, 2, 15, 16, 17, 100, 300])), int(r.choice([0, 1, 4, 16, 17, 130, 1000]))) if r.random() < 0.7 else (0, 0)
        n = max(last + 1, 0)
        seen = np.zeros(n + 1, np.int32)
        steps = L.wenc_selftest_chunk_steps(first, last, window, sinks, step, align, seen.ctypes.data, n)
        pos, key = np.arange(first, last + 1)[:, None], np.arange(n)[None]
        sees = key <= pos
        if window:
            sees &= (key > pos - window) | (key < sinks)
        want = sees.any(0).astype(np.int32)
        # (keys below `sinks` that lie behind every token's window are seen as far as a token stands at or behind them)
        assert np.array_equal(seen[:n], want), (first, last, window, sinks)
        assert steps <= want.sum() // step + 3


@pytest.mark.parametrize("page", [1, 8, 16, 24])
def test_what_a_sequence_gives_back(L, page):
    r = np.random.default_rng(page)
    for _ in range(400):
        length, finished = int(r.integers(0, 300)), bool(r.random() < 0.3)
        window, sinks = (int(r.integers(1, 150)), int(r.choice([0, 1, 4, 40]))) if r.random() < 0.7 else (0, 0)
        total = -(-length // page)
        stay = [e for e in range(total) if e * page < sinks]  # while the sequence does
        # entries none of whose keys the next token sees, nor a later one
        past = [e for e in range(total) if window and (e + 1) * page - 1 <= length - window]
        gone = int(r.integers(0, len(past) + 1))  # what earlier calls gave back
        held = [e for e in range(total) if e >= gone or e in stay]
        want = held if finished else [e for e in past if e >= gone and e not in stay]
        out = np.full(5, -7, np.int32)
        L.wenc_selftest_gives(length, finished, gone, window, sinks, page, out.ctypes.data)
        assert list(range(out[0], out[1])) + list(range(out[2], out[3])) == want
        assert out[4] == (0 if finished else len(past))
