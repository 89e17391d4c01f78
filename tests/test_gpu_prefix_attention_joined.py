"""wenc_prefix_attention in the form that joins partial results (many rows per key head): what a row gives does not
depend on how many rows it shares its prefix with.

The bound is that of the one-launch form for both types (the derivation is in test_gpu_prefix_attention.py): for bf16
  |err| <= 2^-8 |o| + (2 e + 2^-16 + 2 n 2^-23) sum_j p_j |v_j|,  e = 1.1 d + 2^-16 + 2^-21,
with 2^-16 for two-part probabilities. Of some 10^5 elements hundreds are so near zero that the last term is most of
their bound; probabilities held in one bf16 number (2^-9 each, over the square root of the keys) pass it there.
"""
import numpy as np
import pytest

from oracle import decode
from test_gpu_prefix_attention import Case, _joins

pytestmark = pytest.mark.gpu


def _check_two_parts(c, out):
    got = out.double().cpu().numpy()
    ref, absv, A = decode.prefix_attention(c.q.astype(np.float64), c.prefixes, c.owns, c.groups, 0.125)
    keys = max(p[0].shape[0] for p in c.prefixes) + max(o[0].shape[0] for o in c.owns)
    e = 2.0 ** -16 + 2.0 ** -21 + 1.1 * A[..., None] * 0.125 * 64 * 2.0 ** -23
    bound = 2.0 ** -8 * np.abs(ref) + (2 * e + 2.0 ** -16 + 2 * keys * 2.0 ** -23) * absv
    assert np.isfinite(got).all()
    worst = float((np.abs(got - ref) / bound).max())
    assert worst <= 1, f"{worst:.2f} x the bound"


@pytest.mark.parametrize("H,Hkv,q_len,sizes,pre", [
    (32, 32, 1, [160], [129]), (96, 32, 1, [60, 5], [257, 40]), (40, 1, 1, [130, 2], [300, 64]), (4, 4, 7, [40, 180], [500, 127]),
    (1, 1, 1, [2500], [1700])])
def test_probabilities_keep_two_parts_with_many_rows(H, Hkv, q_len, sizes, pre):
    """(with one-part probabilities the first four reached 3.4 to 5.2 times this bound)"""
    c = Case("bf16", sizes, q_len, H, Hkv, pre, None, uneven=len(sizes) > 1, seed=H + q_len, prefix_max=max(pre) + 37)
    assert _joins(c)
    _check_two_parts(c, c.run())
