"""Buffers of the decode-side calls that may not overlap, refused on the host."""
import ctypes

from test_decode_refusals import L, _append  # noqa: F401 (L: a fixture)


def test_queries_in_place_have_one_stride(L):  # noqa: F811
    """In place with two strides, one token's rows would be written over another's before they are read."""
    for kw in (dict(q_stride=512, q_out_stride=576), dict(q_stride=1024, q_out_stride=512), dict(inv_freq=None, q_out_stride=1024)):
        assert L.wenc_kv_append(ctypes.byref(_append(**kw)), None) == 1
        assert b"in place" in L.wenc_last_error()
    assert L.wenc_kv_append(ctypes.byref(_append(n_tokens=0, q_out_stride=576)), None) in (0, 1)
