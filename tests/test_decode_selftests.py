"""The index and angle arithmetic of the decode-side kernels, compiled for the host from the header that the kernels
include, against plain definitions: a token's sequence, the angle that its sine and cosine take, and the runs of key steps
that warps take. A change to that code shows here without a GPU."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

from test_gpu_append_angles import _pi


@pytest.fixture(scope="module")
def L():
    from transformer_encoder_gb300 import lib
    from transformer_encoder_gb300.build import build
    build()
    return lib()


def _sequence(L, start, t, first=None, rows=2 ** 31 - 1):
    start = np.ascontiguousarray(start, np.int32)
    left = ctypes.c_int(-7)
    s = L.wenc_selftest_append_sequence(start.ctypes.data, len(start) - 1, rows, t if first is None else first, t, ctypes.byref(left))
    return s, left.value


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 1000, 1025, 33000])
def test_a_tokens_sequence(L, n):
    """Empty sequences among them; rows behind the last; a warp's run of rows is searched from its first one."""
    r = np.random.default_rng(n)
    start = np.concatenate([[0], np.cumsum(r.integers(0, 3, n))])
    total = int(start[-1])
    for t in r.integers(0, total + 3, 50).tolist() + [0, max(0, total - 1), total, total + 40]:
        want = int(np.searchsorted(start, t, side="right")) - 1
        for first in {t, max(0, t - 1), max(0, t - 7)}:
            s, left = _sequence(L, start, t, first)
            assert s == want if t < total else s == n
            if t < total:
                assert left == start[s + 1] - t


def test_a_sequence_that_ends_behind_the_rows(L):
    start = [0, 3, 3, 10]
    assert _sequence(L, start, 2, rows=9) == (0, 1)
    assert _sequence(L, start, 3, rows=9)[0] == -1
    assert _sequence(L, start, 3, rows=10) == (2, 7)
    assert _sequence(L, start, 10, rows=11)[0] == 3


def test_offsets_out_of_range(L):
    assert _sequence(L, [5, 9], 4)[0] == -1  # they do not start at 0
    assert _sequence(L, [0, 4, 2, 9], 3) in ((0, 1), (2, 6))  # both hold row 3
    r = np.random.default_rng(1)
    for n in (1, 7, 40, 100, 1500):
        for _ in range(50):
            start = r.integers(-2 ** 31, 2 ** 31, n + 1)
            t = int(r.integers(0, 2 ** 31))
            s, _ = _sequence(L, start, t)
            assert -1 <= s <= n
            assert s in (-1, n) or start[s] <= t < start[s + 1]


@pytest.mark.parametrize("f", [1.0, 0.5, 1e-4, 0.31622776, 3.1415927, 6.2831855, 100.0, -0.3, -1e-4, 0.0, 1e-30, 7.5, 1e6, -16777213.0])
@pytest.mark.parametrize("pos", [0, 1, -1, 4095, 1 << 20, (1 << 31) - 1, -1000, -(1 << 31)])
def test_angles(L, f, pos):
    """pi h + l is the position times the frequency modulo a turn. The fraction of a turn for one position is off by at
    most 2^-63 + |f| 2^-84 (two truncations to 2^-64; c2 rounded by 2^-85 and its product by half a step, times |f|),
    l leaves out less than 2^-56 of a turn, and is itself off by 2^-23 of less than 2^-21 as an angle."""
    h, l = ctypes.c_float(), ctypes.c_float()
    L.wenc_selftest_append_angle(f, pos, ctypes.byref(h), ctypes.byref(l))
    h, l = h.value, l.value
    assert -1.0 <= h < 1.0 and 0.0 <= l < 2.0 ** -21
    assert (h * 2 ** 23) % 1 == 0  # 24 bits: exact
    pi = Fraction(_pi(), 1 << 256)
    f = abs(Fraction(float(np.float32(f)))) * (1 if f > 0 else -1)
    off = (Fraction(h) + Fraction(l) / pi - f * pos / pi) % 2  # in half turns
    off = min(off, 2 - off)
    assert off <= 2 * (max(abs(pos), 1) * (Fraction(1, 2 ** 63) + abs(f) / 2 ** 84) + Fraction(1, 2 ** 56)) + Fraction(1, 2 ** 44)


@pytest.mark.parametrize("parts", [1, 4, 8, 32, 64])
def test_runs_score_every_key_once(L, parts):
    r = np.random.default_rng(parts)
    for _ in range(60):
        own = r.integers(0, 60, r.integers(0, 17)).astype(np.int32)
        prefix = int(r.integers(0, 200)) * int(r.integers(0, 2))
        seen = np.zeros(prefix + int(own.sum()) + 16, np.int32)
        L.wenc_selftest_attention_runs(prefix, own.ctypes.data, len(own), parts, seen.ctypes.data)
        assert (seen[:-16] == 1).all() and (seen[-16:] == 0).all()
