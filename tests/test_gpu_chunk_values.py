"""Chunk attention where values and scores that are no numbers meet rows that see no key, or nothing else, and long caches.

Bounds: rows that do not see a bad value are formed from the same keys a second way at most. Each result lies within the
bound of test_gpu_chunk_attention.py of one value: 2^-8 of it for bf16's rounding and, for some hundred keys and weighted
magnitudes below 4, less than 2^-13 times these (float32: 2^-16). Two results differ by twice that.
"""
import pytest

from test_gpu_chunk_attention import Case, plain

pytestmark = pytest.mark.gpu

# [dtype, new tokens, heads, key heads, wide]: tiles of 8, 16 and 32 rows on mma.sync, of one CTA and of clusters, and the tensor
# cores' form with units that are whole within a CTA's run and units that are cut
FORMS = [(dtype, new, H, kv, wide) for dtype in ("bf16", "f32") for new, H, kv in (([4, 8], 4, 4), ([8, 3], 4, 2), ([30, 9], 4, 4))
         for wide in (False, True)] + [("bf16", [256, 300], 40, 40, True), ("bf16", [600, 70], 20, 4, True)]


def near(got, clean, dtype):
    far = clean.float()
    slack = 2.0 ** -7 * far.abs() + 4 * 2.0 ** -12 if dtype == "bf16" else 4 * 2.0 ** -15
    return bool(((got.float() - far).abs() <= slack).all())


@pytest.mark.parametrize("dtype,new,H,kv,wide", FORMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["v", "k"])
def test_rows_without_a_key_beside_rows_that_see_no_number(dtype, new, H, kv, wide, bad, what):
    """Tokens in front of the cache give zeros, whatever the other rows of their tile see."""
    import torch
    lens = [max(1, (5 * m) // 8) for m in new]
    c = Case(dtype, new, [0] * len(new), H, kv, seed=sum(new), wide=wide)
    c.tlens.copy_(torch.tensor(lens, dtype=torch.int32))
    clean = c.run()
    for s, n in enumerate(lens):
        for key in sorted({0, n // 2, n - 1}):
            d = Case(dtype, new, [0] * len(new), H, kv, seed=sum(new), wide=wide)
            d.tlens.copy_(c.tlens)
            (d.vc if what == "v" else d.kc)[int(d.table[s, key // 16]), key % 16, :, 9] = bad
            got = d.run()
            for x, (m, v) in enumerate(zip(new, lens)):
                rows, pos = got[int(c.start[x]):int(c.start[x + 1])], torch.arange(v - m, v, device="cuda")
                assert (rows[pos < 0] == 0).all(), (s, key, x)
                sees = pos >= key if x == s else torch.zeros_like(pos, dtype=torch.bool)
                base = clean[int(c.start[x]):int(c.start[x + 1])]
                assert near(rows[~sees], base[~sees], dtype), (s, key, x)
                if what == "v":
                    hit = rows[sees][..., 9]
                    assert (torch.isnan(hit) if bad != bad else hit == bad).all(), (s, key, x)
                    rest = [e for e in range(64) if e != 9]
                    assert near(rows[sees][..., rest], base[sees][..., rest], dtype), (s, key, x)
                elif bad != bad:
                    assert torch.isnan(rows[sees]).all(), (s, key, x)


@pytest.mark.parametrize("dtype,new,H,kv,wide", FORMS)
@pytest.mark.parametrize("window", [0, 1])
def test_rows_whose_every_score_is_minus_infinity(dtype, new, H, kv, wide, window):
    """exp(s - max s) of nothing but -inf is no number, and neither is the row; a row that sees one other key gives that key no
    weight. (A row that sees no key at all gives zeros.)"""
    import torch
    c = Case(dtype, new, [0] * len(new), H, kv, window=window, seed=sum(new) + 1, wide=wide)
    c.q[..., 9] = c.q[..., 9].abs() + 0.5
    A = c.reference()[2]
    at = [m // 2 if window else 0 for m in new]
    for s, key in enumerate(at):
        c.kc[int(c.table[s, key // 16]), key % 16, :, 9] = -float("inf")
        c.keys[s][0][key, :, 9] = -float("inf")
    got = c.run().double()
    keys = max(new)
    # (the bounds of test_gpu_chunk_attention.py; A without the infinite scores, whose weights are zeros exactly)
    for s, (m, key) in enumerate(zip(new, at)):
        rows = slice(int(c.start[s]), int(c.start[s + 1]))
        ref, absv, _ = plain(c.q[rows].double(), *c.keys[s], torch.arange(m, device="cuda"), window, 0, 0.125)
        assert torch.isnan(ref[key]).all() and torch.isnan(got[rows][key]).all(), s
        rest = [i for i in range(m) if i != key]
        e = 2.0 ** -16 + 2.0 ** -21
        if dtype == "bf16":
            e = e + 1.1 * A[rows][rest] * 64 * 2.0 ** -23
            bound = 2.0 ** -8 * ref[rest].abs() + (2 * e + 2.0 ** -16 + 2 * keys * 2.0 ** -23) * absv[rest]
        else:
            e = e + 1.1 * A[rows][rest] * (3 * 2.0 ** -22 + 192 * 2.0 ** -23)
            bound = 2.0 ** -24 * ref[rest].abs() + (2 * e + 3 * 2.0 ** -22 + 4 * keys * 2.0 ** -23) * absv[rest]
        err = (got[rows][rest] - ref[rest]).abs()
        assert (err <= bound + 1e-30).all(), (s, float((err / (bound + 1e-30)).max()))


def test_no_wait_runs_out_while_rows_are_formed_again():
    """A value that is no number in a cache of 60000 keys, seen by rows of two units that lie whole in a CTA's run, with more of the
    run behind them: those rows take a second evaluation over all their keys, which no role of the kernel may wait for. The
    error word stays clear (run() reads it), and rows that do not see the value keep theirs."""
    import torch
    m, n, H, window = 1000, 61000, 128, 59000  # one key head: units of two tokens, 463 steps each, some three units a CTA
    case = dict(dtype="bf16", new=[m], past=[n - m], H=H, Hkv=1, window=window, sinks=0, page=64, seed=21)
    c = Case(**case)
    clean = c.run()
    key = n - m - window + 3  # in the windows of the first three tokens alone
    pos = torch.arange(n - m, n, device="cuda")
    sees = (key <= pos) & (key > pos - window)
    assert sees.nonzero().flatten().tolist() == [0, 1, 2]
    c.vc[int(c.table[0, key // 64]), key % 64, 0, 9] = float("nan")
    got = c.run()
    # (units of which no row sees the value: the same bits)
    assert torch.equal(got[4:], clean[4:])
    assert torch.isnan(got[:3, :, 9]).all()
    # Elsewhere both results lie within the bound of test_gpu_chunk_attention.py of one value: its d with A < 64 (|q . k| sums
    # of 64 products of unit normals), 59000 keys, weighted magnitudes below 1; and as there 2^-8 each over all elements.
    e = 1.1 * 64 * 64 * 2.0 ** -23 + 2.0 ** -16 + 2.0 ** -21
    seen = torch.ones_like(got[:4], dtype=torch.bool)
    seen[:3, :, 9] = False
    far, err = clean[:4][seen].double(), (got[:4][seen].double() - clean[:4][seen].double())
    assert (err.abs() <= 2.0 ** -7 * far.abs() + 2 * (2 * e + 2.0 ** -16 + 2 * window * 2.0 ** -23)).all()
    assert float(err.norm()) <= 2.0 ** -7 * float(far.norm())
