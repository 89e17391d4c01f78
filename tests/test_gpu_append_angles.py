"""The sines and cosines of wenc_kv_append: a key of pairs (1, 0) turns to (cos, sin) of its angle, exactly as held.

Bound. The angle is a 64-bit fraction of a turn of two truncated parts, off by at most |P| * 3 * 2^-64 turns for position P (< |P| *
2^-59 as an angle). Its leading 24 bits are exact in sincospif, whose stated error is one unit in the last place (2^-23 of
the value); the rest l < 2^-21 enters to first order (l^2 / 2 < 2^-43), with its own roundings (2^-44), and the sum
rounds once (2^-24): |err| <= 1.5 * 2^-23 |value| + 2^-42 + |P| 2^-59. (An angle of 24 bits is off by up to 1.5 * 2^-24, which is
more than that wherever a sine or cosine is small.)
"""
from fractions import Fraction

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _pi(bits=256):
    """floor(pi 2^bits), by Machin's formula."""
    one = 1 << (bits + 16)

    def arctan_inv(x):
        total, term, n = 0, one // x, 1
        while term:
            total += term // n if n % 4 == 1 else -(term // n)
            term //= x * x
            n += 2
        return total

    return 4 * (4 * arctan_inv(5) - arctan_inv(239)) >> 16


def _cos_sin(pos, freq):
    """cos and sin of pos * freq to some 2^-52: the angle less its nearest multiple of pi, in integers of 256 bits."""
    pi, bits = _pi(), 256
    c, s = np.zeros((len(pos), len(freq))), np.zeros((len(pos), len(freq)))
    for j, f in enumerate(freq):
        f = Fraction(float(f))
        for i, p in enumerate(pos):
            angle = int(p) * f.numerator * (1 << bits) // f.denominator
            n = (2 * angle + pi) // (2 * pi)
            r = float(Fraction(angle - n * pi, 1 << bits))
            c[i, j], s[i, j] = (np.cos(r), np.sin(r)) if n % 2 == 0 else (-np.cos(r), -np.sin(r))
    return c, s


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [16, 64])
@pytest.mark.parametrize("span", [2, 1500, 1 << 20, (1 << 31) - 1])
def test_sines_and_cosines(interleaved, rot, span):
    import torch
    from transformer_encoder_gb300 import kv_append, sync_status
    n, half = 700, rot // 2
    r = np.random.default_rng(span % 1000 + rot)
    pos = r.integers(-span, span + 1, n)
    freq = np.array([10000.0 ** (-2.0 * i / rot) * (-1) ** (i // 3) for i in range(half)], np.float32)
    freq[1], freq[2] = np.float32(np.pi / 7), np.float32(1e-7)  # near multiples of pi, and hardly turning
    k = torch.zeros(n, 1, 64, device="cuda")
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, half), slice(half, rot))
    k[:, :, a] = 1.0
    pages = torch.zeros(2, n, 1, 1, 64, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    kv_append(k, k, pages[0], pages[1], i32([list(range(n))]), i32([n]), positions=i32(pos.tolist()),
              inv_freq=torch.from_numpy(freq).cuda(), interleaved=interleaved)
    sync_status()
    got = pages[0, :, 0, 0].double().cpu().numpy()
    for x, want in zip((got[:, a], got[:, b]), _cos_sin(pos, freq)):
        bound = 1.5 * 2.0 ** -23 * np.abs(want) + 2.0 ** -42 + np.abs(pos)[:, None] * 2.0 ** -59
        worst = float((np.abs(x - want) / bound).max())
        assert worst <= 1, f"{worst:.2f} x the bound"
