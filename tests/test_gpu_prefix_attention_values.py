"""wenc_prefix_attention on values that are no numbers, or hardly one: what a row does not see never reaches it.

Bounds are those of test_gpu_prefix_attention.py. Rows that see a non-finite value take it at its element alone: a NaN
stays one, and an infinity (all weights of these cases are positive and far from underflow) stays that infinity.
"""
import numpy as np
import pytest

from test_gpu_prefix_attention import DTYPES, Case, _joins

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("pre", [50, 0])
@pytest.mark.parametrize("size,q_len", [(3, 1), (3, 3), (70, 1), (70, 3), (3700, 1), (1300, 3)])
def test_values_that_are_no_numbers_reach_those_who_see_them(dtype, bad, pre, size, q_len):
    """One element of one sequence's newest own value: it is the last token's alone, not the older draft tokens', not
    the other sequences' of the group, and not that of a neighbour without own keys."""
    import torch
    own = [9] * size
    own[1] = 0
    c = Case(dtype, [size], q_len, 2, 2, [pre], own, seed=30, page=4)
    if pre:
        assert _joins(c) == (size > 100)
    page, slot = int(c.kw["block_table"][2, 2]), 0  # own key 8 of sequence 2
    clean = c.kw["v_pages"][page, slot, 1, 37].clone()
    c.kw["v_pages"][page, slot, 1, 37] = float(bad)
    out = c.run()
    got = out[2, q_len - 1, 1, 37].item()
    assert np.isnan(got) if bad == "nan" else got == float(bad)
    c.kw["v_pages"][page, slot, 1, 37] = clean
    out[2, q_len - 1, 1, 37] = c.run()[2, q_len - 1, 1, 37]
    c.check(out)  # every other element
    if pre == 0:
        assert (out[1] == 0).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [3, 70])
def test_infinite_prefix_values_stay_infinite_in_the_one_launch_form(dtype, size):
    import torch
    c = Case(dtype, [size], 1, 2, 2, [50], [9] * size, seed=31)
    assert not _joins(c)
    want = c.run()
    c.kw["v_prefix"][0, 20, 1, 5] = float("inf")
    out = c.run()
    assert (out[:, 0, 1, 5] == float("inf")).all()
    out[:, 0, 1, 5] = want[:, 0, 1, 5]
    assert torch.equal(out, want)


@pytest.mark.parametrize("size", [3, 70, 3700])
def test_values_near_the_largest_number(size):
    """fp32 numbers within 2^-12 of the largest one: rounding one to fewer bits would leave the range. As values: the
    result is half of it, by two keys of equal weight, the other's value 0. As keys of queries of zeros, and as queries of
    keys of zeros: they weigh like any other."""
    import torch
    c = Case("f32", [size], 1, 2, 2, [1], [1] * size, seed=32)
    assert _joins(c) == (size == 3700)
    big = torch.finfo(torch.float32).max
    c.tq.zero_()
    for where, zero in ((c.kw["v_prefix"], c.kw["v_pages"]), (c.kw["v_pages"], c.kw["v_prefix"])):
        where.fill_(big)
        zero.fill_(0.0)
        out = c.run()
        # 2^-21 of a product of parts, 2^-24 of the output, and the sums'
        assert ((out - big / 2).abs() <= 2.0 ** -19 * big).all()
    want = out
    for where in (c.kw["k_prefix"], c.kw["k_pages"], c.tq):
        for t in (c.kw["k_prefix"], c.kw["k_pages"], c.tq):
            t.zero_()
        where.fill_(big)
        assert ((c.run() - want).abs() <= 2.0 ** -19 * big).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,sizes", [(2, [3, 2]), (32, [160, 90])])
def test_a_prefix_of_no_tokens(dtype, H, sizes):
    """As one of length zero: the own keys alone, zeros where there are none, and rows of no group as they were."""
    import torch
    r = np.random.default_rng(H)
    c = Case(dtype, sizes, 2, H, H, [0, 0], [int(x) for x in r.integers(0, 20, sum(sizes) + 3)], uneven=True, extra=3, seed=33)
    side = torch.cuda.Stream()
    want = torch.full_like(c.tq, 7.0)
    c.check(c.run(out=want))
    for name in ("k_prefix", "v_prefix"):
        c.kw[name] = c.kw[name][:, :0]
    for kw in (dict(), dict(stream=side)):
        for lens in (c.kw["prefix_lens"], None):
            c.kw["prefix_lens"] = lens
            out = torch.full_like(c.tq, 7.0)
            side.wait_stream(torch.cuda.current_stream())
            c.run(out=out, **kw)
            assert torch.equal(out, want)
        c.kw["prefix_lens"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    del c.kw["k_pages"], c.kw["v_pages"], c.kw["lens"], c.kw["block_table"]
    assert (c.run()[:sum(sizes)] == 0).all()
