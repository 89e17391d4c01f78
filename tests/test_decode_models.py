"""CPU models of the index and angle arithmetic inside the decode-side kernels, against plain
definitions: the search for a token's sequence, the runs of key steps that warps take, and the 64-bit
fractions of a turn. Each model follows the kernel's code line by line."""
from fractions import Fraction

import numpy as np
import pytest


# ------------------------------------------------------------------ append.cu, find_seq
def find_seq(start, t):
    """The last index with start[i] <= t (-1: none), 32 probes a step."""
    lo, length = 0, len(start)
    while length > 0:
        step = (length + 31) // 32
        hits = 0
        for lane in range(32):
            if lane * step < length:
                assert 0 <= lo + lane * step < len(start)  # every probe inside the array
                hits += start[lo + lane * step] <= t
        if hits == 0:
            return lo - 1
        base = (hits - 1) * step
        rest = min(step, length - base) - 1
        lo += base + 1
        length = rest
    return lo - 1


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 1000, 1025, 33000])
def test_sequence_search(n):
    r = np.random.default_rng(n)
    start = np.concatenate([[0], np.cumsum(r.integers(0, 3, n))])  # empty sequences among them
    for t in r.integers(0, start[-1] + 3, 50).tolist() + [0, int(start[-1]) - 1, int(start[-1])]:
        if t >= 0:
            assert find_seq(start, t) == int(np.searchsorted(start, t, side="right")) - 1
    assert find_seq(start + 5, 4) == -1


def test_sequence_search_stays_inside_any_array():
    """Offsets that do not ascend give some index of the array, never a probe outside it."""
    r = np.random.default_rng(1)
    for n in (1, 7, 40, 100, 1500):
        for _ in range(20):
            start = r.integers(-2 ** 31, 2 ** 31, n + 1)
            assert -1 <= find_seq(start, int(r.integers(-2 ** 31, 2 ** 31))) <= n


# ------------------------------------------------------------------ append.cu, turns64
TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965068423413596")


def turns64(f):
    """The kernel's double arithmetic on one fp32 frequency."""
    c1, c2 = float.fromhex("0x1.45f306dp-3"), float.fromhex("0x1.9391054a7f09dp-32")
    hi, lo = abs(float(np.float32(f))) * c1, abs(float(np.float32(f))) * c2
    hi -= np.floor(hi)
    h32 = hi * 4294967296.0
    top = int(h32)
    low = int((h32 - float(top)) * 4294967296.0)
    lo -= np.floor(lo)
    l32 = lo * 4294967296.0
    ltop = int(l32)
    llow = int((l32 - float(ltop)) * 4294967296.0)
    turn = (top << 32) + low + (ltop << 32) + llow
    return (-turn if f < 0 else turn) % 2 ** 64


@pytest.mark.parametrize("f", [1.0, 0.5, 1e-4, 0.31622776, 3.1415927, 6.2831855, 100.0, -0.3, -1e-4, 0.0, 1e-30, 7.5, 1e6, -16777213.0])
@pytest.mark.parametrize("pos", [0, 1, 4095, 1 << 20, (1 << 31) - 1, -1000, -(1 << 31)])
def test_angles_are_exact_modulo_a_turn(f, pos):
    """position * frequency / 2 pi modulo 1 to 2^-31 of a turn (what the single-precision sine is
    given), for every position of 32 bits. The fraction is off by at most 2^-63 + |f| 2^-84: its two
    truncations to 2^-64; c2 in [2^-32, 2^-31) is rounded by at most 2^-85, times |f|; the product
    f c2 < |f| 2^-31 by half a step, at most |f| 2^-31 2^-53. That is below 2^-62 for |f| <= 2^20."""
    got = Fraction(turns64(f) * pos % 2 ** 64, 2 ** 64)
    want = Fraction(float(np.float32(f))) * pos / TWO_PI
    off = (got - want) % 1
    off = min(off, 1 - off)
    assert off <= max(abs(pos), 1) * (Fraction(1, 2 ** 63) + abs(Fraction(float(np.float32(f)))) / 2 ** 84)
    signed = turns64(f) * pos % 2 ** 64
    signed -= 2 ** 64 if signed >= 2 ** 63 else 0
    top = np.float32(signed >> 32) * np.float32(2.0 ** -31)  # sincospi's argument, in half turns
    diff = (Fraction(float(top)) / 2 - want) % 1
    assert min(diff, 1 - diff) <= Fraction(1, 2 ** 25)


# ------------------------------------------------------------------ prefix_attn.cu, segments and runs
def steps_of(prefix_len, own):
    step0, lens = [0, (prefix_len + 15) // 16], [prefix_len]
    for n in own:
        step0.append(step0[-1] + (n + 15) // 16)
        lens.append(n)
    return step0, lens


@pytest.mark.parametrize("parts", [1, 4, 8, 32, 64])
def test_runs_cover_every_key_once(parts):
    """Every key of every segment is scored by exactly one warp, for lengths with zeros among them."""
    r = np.random.default_rng(parts)
    for _ in range(40):
        own = [int(x) for x in r.integers(0, 60, r.integers(0, 17))]
        prefix = int(r.integers(0, 200)) * int(r.integers(0, 2))
        step0, lens = steps_of(prefix, own)
        n = step0[1 + len(own)]
        per = (n + parts - 1) // parts
        seen = [np.zeros(m, int) for m in lens]
        for part in range(parts):
            first, count = part * per, max(0, min(per, n - part * per))
            seg = 0
            for t in range(first, first + count):
                while t >= step0[seg + 1]:
                    seg += 1
                    assert seg < len(lens)  # the walk ends inside the table
                key0 = (t - step0[seg]) * 16
                assert key0 < lens[seg]
                seen[seg][key0:key0 + 16] += 1
        assert all((s == 1).all() for s in seen)
