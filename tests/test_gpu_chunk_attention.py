"""wenc_chunk_attention against its float64 definition, at the sizes, windows and lengths where it can go wrong.

Bounds, from the arithmetic. Let A = max_j sum_i |q_i k_ij| of the row and n the keys it sees.
bf16: products of bf16 are exact in fp32; 64 of them accumulate with at most 64 roundings of 2^-23
relative to A each (the tensor core may truncate), so a score is off by d = scale * A * 64 * 2^-23,
plus two roundings of the exponent's argument (at most 2 * 128 * 2^-24 = 2^-16 in log2 units: inputs
are scaled so that |argument| < 128) and 2^-21 for exp2: p is off by e = 1.1 d + 2^-16 + 2^-21
relative, numerator and denominator both. P enters the product as two bf16 parts: 2^-16 more in the
numerator. Sums over n keys: n * 2^-23 each. Output rounding: 2^-8 (half a step of bf16).
  |err| <= 2^-8 |o| + (2 e + 2^-16 + 2 n 2^-23) sum_j p_j |v_j|
fp32: every operand is two TF32 parts that miss it by less than 2^-22 (11 bits rounded, 11 more of the rest cut
off), the product of the small parts (2^-11 each) is dropped: 3 * 2^-22 a product, and three times as many
accumulations; output 2^-24:
  d = scale * A * (3 * 2^-22 + 192 * 2^-23), and in the numerator 3 * 2^-22 + 4 n 2^-23.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

DTYPES = ["bf16", "f32"]


def plain(q, k, v, pos, window, sinks, scale):
    """(out, sum_j p_j |v_j|, A) in 64 bits of the tokens q [m, H, 64] at positions pos of one sequence with keys k and v
    [len, Hkv, 64]."""
    import torch
    m, H, _ = q.shape
    n, kv, _ = k.shape
    out, absv, A = (torch.zeros(m, H, 64, dtype=torch.float64, device=q.device) for _ in range(3))
    j, p = torch.arange(n, device=q.device).view(1, n), pos.view(m, 1)
    sees = j <= p
    if window:
        sees &= (j > p - window) | (j < sinks)
    some = sees.any(1, keepdim=True)
    for h in range(H if n else 0):
        kh, vh = k[:, h // (H // kv)], v[:, h // (H // kv)]
        s = (q[:, h] @ kh.t() * scale).masked_fill(~sees, -torch.inf)
        w = torch.softmax(s.masked_fill(~some, 0.0), 1) * some
        w = w.masked_fill(~sees, 0.0)
        out[:, h], absv[:, h] = w @ vh, w @ vh.abs()
        A[:, h] = ((q[:, h].abs() @ kh.abs().t()) * sees).amax(1, keepdim=True) * abs(scale)
    return out, absv, A


class Case:
    """One problem. Keys that no token sees, and pages without one, hold NaN; so do padding rows of q. wide: a block table for
    caches so long that the call is not taken for a little one, and its long chunks go to the tensor cores' form (bf16)."""

    def __init__(self, dtype, new, past, H, Hkv, window=0, sinks=0, page=16, pad=0, strided=False, seed=0, extra_pages=3, odd_pages=False,
                 wide=False):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = np.random.default_rng(seed)
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.dtype, self.new, self.lens, self.H, self.Hkv = dtype, list(new), [a + b for a, b in zip(new, past)], H, Hkv
        self.window, self.sinks, self.page = window, sinks, page
        self.start = np.cumsum([0] + self.new)
        rows = int(self.start[-1]) + pad
        around = torch.full((rows, H + 3, 64), float("nan"), device="cuda", dtype=self.dt)
        q = torch.randn(rows, H, 64, generator=g, device="cuda").to(self.dt)
        q[int(self.start[-1]):] = float("nan")
        if strided:
            around[:, 1:1 + H] = q
            q = around[:, 1:1 + H]
        self.q = q
        need = [-(-n // page) for n in self.lens]
        total, width = max(1, sum(need)) + extra_pages, max(1, max(need)) + (4096 if wide else 1)
        order = r.permutation(total)
        shape = (total, page, Hkv, 64)
        self.kc, self.vc = (torch.full(shape, float("nan"), device="cuda", dtype=self.dt) for _ in range(2))
        if odd_pages:  # pages further apart than they are long, keys and values differently
            self.kc = torch.full((total, page + 1, Hkv, 64), float("nan"), device="cuda", dtype=self.dt)[:, :page]
            self.vc = torch.full((total, 2 * page + 3, Hkv, 64), float("nan"), device="cuda", dtype=self.dt)[:, 1:1 + page]
        table = np.full((len(new), width), -1, np.int32)
        self.keys, at = [], 0
        for s, (m, n) in enumerate(zip(self.new, self.lens)):
            k, v = (torch.randn(n, Hkv, 64, generator=g, device="cuda").to(self.dt) for _ in range(2))
            seen = np.zeros(n, bool)
            for p in range(max(n - m, 0), n):
                seen[max(0, p - window + 1) if window else 0:p + 1] = True
                seen[:min(sinks, p + 1)] |= window > 0
            mine = order[at:at + need[s]]
            at += need[s]
            keep = [bool(seen[e * page:(e + 1) * page].any()) for e in range(need[s])]
            table[s, :need[s]] = np.where(keep, mine, -1 if s % 2 else total + 7)  # (pages that are gone: any number)
            idx = torch.from_numpy(np.flatnonzero(seen)).cuda()
            if idx.numel():
                pages = torch.from_numpy(mine).cuda()[idx // page]
                self.kc[pages, idx % page], self.vc[pages, idx % page] = k[idx], v[idx]
            self.keys.append((k.double(), v.double()))
        self.table = torch.from_numpy(table).cuda()
        self.tlens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.tstart = torch.tensor(self.start.tolist(), dtype=torch.int32, device="cuda")

    def run(self, **kw):
        from transformer_encoder_gb300 import chunk_attention, sync_status
        kw = {"seq_start": self.tstart, "max_new": max(1, max(self.new)), "window": self.window or None, "sinks": self.sinks, **kw}
        out = chunk_attention(self.q, self.kc, self.vc, self.table, self.tlens, **kw)
        sync_status()
        return out

    def reference(self, scale=0.125):
        import torch
        parts = []
        for s, (m, n) in enumerate(zip(self.new, self.lens)):
            q = self.q[int(self.start[s]):int(self.start[s]) + m].double()
            parts.append(plain(q, *self.keys[s], torch.arange(n - m, n, device="cuda"), self.window, self.sinks, scale))
        return [torch.cat(x) for x in zip(*parts)]

    def check(self, out, scale=0.125, what=""):
        import torch
        n = int(self.start[-1])
        got = out[:n].double()
        ref, absv, A = self.reference(scale)
        assert (1.4427 * A < 128).all()
        keys = max(self.lens + [1])
        e = 2.0 ** -16 + 2.0 ** -21
        if self.dtype == "bf16":
            e = e + 1.1 * A * 64 * 2.0 ** -23
            bound = 2.0 ** -8 * ref.abs() + (2 * e + 2.0 ** -16 + 2 * keys * 2.0 ** -23) * absv
        else:
            e = e + 1.1 * A * (3 * 2.0 ** -22 + 192 * 2.0 ** -23)
            bound = 2.0 ** -24 * ref.abs() + (2 * e + 3 * 2.0 ** -22 + 4 * keys * 2.0 ** -23) * absv
        assert torch.isfinite(got).all(), what
        err = (got - ref).abs()
        assert (err <= bound + 1e-30).all(), f"{what}: {float((err / (bound + 1e-30)).max()):.2f} x the bound"
        if float(ref.norm()) > 0:  # what a systematic mistake under the elementwise bound would show
            assert float((got - ref).norm()) <= (2.0 ** -8 if self.dtype == "bf16" else 2.0 ** -19) * float(ref.norm()), what


def _ints(seed, n, lo, hi):
    return [int(x) for x in np.random.default_rng(seed).integers(lo, hi, n)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("past", [0, 1, 14, 15, 16, 31, 127, 128, 300])
@pytest.mark.parametrize("page", [1, 3, 16, 64])
def test_single_tokens(dtype, past, page):
    """Lengths from one on that end inside a page and a step, an empty sequence among them."""
    c = Case(dtype, [1, 0, 1], [past, 5, past // 2], 4, 2, page=page, seed=past * 7 + page)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 0), (100, 4), (100, 40), (64, 200), (5000, 3)])
@pytest.mark.parametrize("new", [1, 5, 70])
def test_windows_and_sinks(dtype, window, sinks, new):
    """Windows shorter and longer than the keys, sinks that meet the window, pages behind it that are gone."""
    c = Case(dtype, [new, new, 1], [1000, 90, 333], 4, 4, window, sinks, page=8, seed=window + sinks)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 6), (20, 4), (5, 1), (16, 2), (40, 1)])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("wide", [False, True])
def test_head_layouts_of_ragged_chunks(dtype, H, Hkv, window, wide):
    """Chunks of every size in one call, padding rows behind them that stay as they are."""
    import torch
    new = [1, 0, 2, 130, 1, 33, 7, 1, 257, 0]
    c = Case(dtype, new, _ints(H, len(new), 0, 300), H, Hkv, window, 3 if window else 0, page=24, pad=9, strided=H == 6, seed=H, wide=wide)
    out = torch.full(c.q.shape, 7.0, device="cuda", dtype=c.dt)
    assert c.run(out=out) is out
    c.check(out)
    assert (out[sum(new):] == 7.0).all()
    fresh = c.run()
    assert torch.equal(fresh[:sum(new)], out[:sum(new)]) and (fresh[sum(new):] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,past", [([300], [0]), ([511, 129], [700, 5]), ([64, 64, 64], [64, 2000, 0]), ([1000], [3000])])
@pytest.mark.parametrize("H,Hkv", [(4, 4), (10, 2)])
@pytest.mark.parametrize("wide", [False, True])
def test_prompts(dtype, new, past, H, Hkv, wide):
    """Many tokens of one sequence: rows over several tiles, keys from a prompt's first to those of a long cache."""
    c = Case(dtype, new, past, H, Hkv, page=16, seed=sum(new), wide=wide)
    c.check(c.run())


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 0), (100, 40), (64, 200), (128, 0), (5000, 3)])
def test_windows_of_many_rows(window, sinks):
    """The same borders in the tensor cores' form: enough rows that a short window's call is no little one."""
    c = Case("bf16", [300, 70], [1000, 20], 40, 20, window, sinks, page=8, seed=window + sinks)
    c.check(c.run())


@pytest.mark.parametrize("page", [1, 3, 24, 100])
def test_pages_of_many_rows(page):
    c = Case("bf16", [130, 1, 270], [0, 40, 515], 20, 4, page=page, seed=page, wide=True)
    c.check(c.run())


@pytest.mark.parametrize("H,Hkv", [(128, 1), (130, 1), (66, 1), (3, 1)])
def test_many_query_heads_a_key_head(H, Hkv):
    """One token a row tile, rows that leave most of a tile empty, and more heads than a tile has rows (the other form)."""
    c = Case("bf16", [90, 1, 3], [200, 40, 0], H, Hkv, page=16, seed=H, wide=True)
    c.check(c.run())


@pytest.mark.parametrize("jump", [30.0, 200.0, 3000.0])
def test_scores_that_leave_their_reference_behind(jump):
    """Scores far above those of a row's first keys, suddenly and step by step: the reference that weights are formed against follows."""
    import torch
    c = Case("bf16", [200], [1500], 4, 2, seed=14, wide=True)
    pages = c.table[0, :-(-1700 // 16)].long()
    k = torch.zeros(1712, 2, 64, device="cuda", dtype=torch.bfloat16)
    k[:1700] = c.keys[0][0].to(torch.bfloat16) * 0.25
    # along the mean query, so that every row's scores jump: at key 700, and a little at every 60th
    c.q.fill_(0.25)
    k[700, :, :] += jump / 16
    for i, key in enumerate(range(900, 1690, 60)):
        k[key, 1] += jump / 16 * (1 + i / 8)
    c.kc[pages] = k.view(-1, 16, 2, 64)
    c.keys[0] = (k[:1700].double(), c.keys[0][1])
    out, (ref, absv, _) = c.run().double(), c.reference()
    # The bound above, whose two roundings of the exponent's argument (2^-24 each of up to 1.4427 A) are not held to arguments
    # below 128 here. A <= 64 * 0.25 * (187.5 * 2.625 + 2) * 0.125 < 990, e < 0.01, so first order in e still holds (e^2 < 2^-13 is
    # added).
    _, _, A = c.reference()
    assert (A < 990).all()
    e = 1.1 * A * 64 * 2.0 ** -23 + 2 * 1.4427 * A * 2.0 ** -24 + 2.0 ** -16 + 2.0 ** -21
    bound = 2.0 ** -8 * ref.abs() + (2 * e + 2.0 ** -13 + 2.0 ** -16 + 2 * 1700 * 2.0 ** -23) * absv
    assert torch.isfinite(out).all()
    err = (out - ref).abs()
    assert (err <= bound + 1e-30).all(), float((err / (bound + 1e-30)).max())


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompts_behind_windows(dtype):
    c = Case(dtype, [700, 300, 1], [2500, 40, 900], 6, 2, 333, 5, page=8, seed=4)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
def test_equal_chunks_without_offsets(dtype):
    import torch
    c = Case(dtype, [9] * 6, _ints(2, 6, 0, 200), 8, 4, seed=3)
    out = c.run(seq_start=None, max_new=None)
    c.check(out)
    assert torch.equal(out, c.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m", [1, 4, 70])
def test_a_loose_bound_without_offsets(dtype, m):
    """Sequences of equal chunks, for which the call allows far more tokens than they bring: every row is written."""
    import torch
    c = Case(dtype, [m] * 40, _ints(m, 40, 0, 300), 8, 4, seed=m, wide=True)
    for start in (None, c.tstart):
        out = torch.full(c.q.shape, float("nan"), device="cuda", dtype=c.dt)
        c.check(c.run(seq_start=start, max_new=40 * m, out=out))


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_call_that_allows_chunks_and_gets_none(dtype):
    """Room for long chunks: single tokens alone, then padding alone (rows behind the last sequence stay as they are)."""
    import torch
    c = Case(dtype, [1] * 9 + [0], _ints(1, 10, 0, 400), 20, 4, pad=600, seed=15, wide=True)
    out = torch.full(c.q.shape, 7.0, device="cuda", dtype=c.dt)
    c.check(c.run(max_new=600, out=out))
    assert (out[9:] == 7).all()
    c = Case(dtype, [0] * 3, [5, 0, 90], 20, 4, pad=600, seed=16, wide=True)
    out = torch.full(c.q.shape, 7.0, device="cuda", dtype=c.dt)
    c.run(max_new=600, out=out)
    assert (out == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_chunks_that_lie_in_front_of_the_cache(dtype):
    """Whole runs of tokens at negative positions, a sequence of length 0 among them: rows of zeros."""
    import torch
    c = Case(dtype, [600, 300], [0, 0], 4, 2, seed=17, wide=True)
    c.tlens.copy_(torch.tensor([30, 0], dtype=torch.int32))
    out = c.run(out=torch.full(c.q.shape, 7.0, device="cuda", dtype=c.dt))
    assert (out[:570] == 0).all() and (out[600:] == 0).all()
    assert torch.isfinite(out).all() and (out[570:600] != 7).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", [False, True])
def test_a_bound_on_the_tokens_does_not_change_them(dtype, wide):
    """What a sequence brings decides its results' exactness, not how many the call allows."""
    c = Case(dtype, [1, 3, 200, 12], [500, 60, 10, 4000], 8, 2, seed=5, wide=wide)
    c.check(c.run())
    c.check(c.run(max_new=None))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [1.0 / 64, -0.125, 0.0])
@pytest.mark.parametrize("wide", [False, True])
def test_scales(dtype, scale, wide):
    c = Case(dtype, [1, 40, 200], [300, 70, 90], 4, 2, seed=6, wide=wide)
    c.check(c.run(scale=scale), scale)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", [False, True])
def test_tokens_in_front_of_the_cache_see_nothing(dtype, wide):
    """A length below the tokens that a sequence brings: the first of them stand at negative positions."""
    import torch
    c = Case(dtype, [6, 150], [0, 0], 4, 2, seed=7, wide=wide)
    full = c.reference()[0]
    c.tlens.copy_(torch.tensor([2, 40], dtype=torch.int32))
    out = c.run().double()
    assert (out[:4] == 0).all() and (out[6:116] == 0).all()
    assert not torch.equal(out[4:6], torch.zeros_like(out[4:6])) and torch.isfinite(out).all()
    del full


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,past,H,Hkv", [([1, 1, 8], [200, 30, 100], 4, 2), ([200, 1, 300], [50, 400, 900], 4, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("many", [1, 10])
def test_values_that_are_no_numbers_reach_the_rows_that_see_them(dtype, new, past, H, Hkv, bad, many):
    """A value (and a key) behind a token's own position, or outside its window, leaves its row as it is; the rows that see it take it
    as a plain evaluation does."""
    import torch
    H, Hkv = H * many, Hkv * many  # (with ten times the heads the long chunks are no little call)
    c = Case(dtype, new, past, H, Hkv, 120, 2, page=8, seed=8)
    clean = c.run()
    s, n, m = 2, c.lens[2], new[2]
    others = [e for e in range(64) if e != 9]
    for key in (n - 1, n - m // 2 - 1, 1):
        for what in ("v", "k"):
            if what == "k" and bad == 3e38:
                continue  # (scores of 1e38 are numbers, but none that 32 bits tell apart)
            d = Case(dtype, new, past, H, Hkv, 120, 2, page=8, seed=8)
            page = int(d.table[s, key // 8])
            (d.vc if what == "v" else d.kc)[page, key % 8, 1, 9] = bad
            got = d.run()
            pos = torch.arange(n - m, n, device="cuda")
            sees = (key <= pos) & ((key > pos - 120) | (key < 2))
            rows = torch.zeros(sum(new), H, dtype=torch.bool, device="cuda")
            rows[sum(new[:2]):, H // Hkv:2 * (H // Hkv)] = sees.view(-1, 1)
            # Rows that do not see it keep their values. Not every bit: the element beside the bad value is formed a second way, and a
            # score that moves the running maximum of one row of a tile moves its other rows' references too (to what they are
            # anyway). Both results lie within the bound above of one value: 2^-8 each of it for the rounding; the rest, for
            # some hundred keys, below 2^-13 of the weighted magnitudes, which stay below 4 here (float32: 2^-16).
            near, far = got[~rows].float(), clean[~rows].float()
            slack = 2.0 ** -7 * far.abs() + 4 * 2.0 ** -12 if dtype == "bf16" else torch.full_like(far, 4 * 2.0 ** -15)
            assert ((near - far).abs() <= slack).all(), (key, what)
            hit = got[rows].float()
            if what == "v":
                scale = clean[rows].float().abs().amax()
                assert ((hit[:, others] - clean[rows].float()[:, others]).abs() <= (2.0 ** -7 if dtype == "bf16" else 2.0 ** -17) * scale).all()
                if bad != bad:
                    assert torch.isnan(hit[:, 9]).all()
                elif abs(bad) == float("inf"):
                    assert (hit[:, 9] == bad).all()
                else:
                    assert torch.isfinite(hit[:, 9]).all() and (hit[:, 9] > 1e30).all()
            elif bad != bad:
                assert torch.isnan(hit).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", [False, True])
def test_a_lowest_score_is_no_mask(dtype, wide):
    """Keys whose scores are the type's lowest values for all that a row sees: an even mean, not zeros."""
    import torch
    c = Case(dtype, [3, 150], [40, 3], 2, 2, seed=9, wide=wide)
    c.q[:] = 0
    out = c.run()
    c.check(out)
    c.q.fill_(1.0)
    c.kc.nan_to_num_(0.0).fill_(-2.0 ** 20)  # every score -2^23
    got = c.run().double()
    at = 0
    for s, m in enumerate(c.new):
        n, v = c.lens[s], c.keys[s][1]
        for i in range(m):
            mean = v[:n - m + i + 1].mean(0)
            assert (got[at + i] - mean).abs().max() <= 2.0 ** -8 * mean.abs().max() + 1e-5
        at += m


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", ["page", "length", "long", "offset", "behind", "many"])
@pytest.mark.parametrize("wide", [False, True])
def test_bad_lengths_offsets_and_pages_are_reported(dtype, case, wide):
    """Reported, nothing out of range accessed, and the other sequences right."""
    import torch
    from transformer_encoder_gb300 import WencError, sync_status
    c = Case(dtype, [1, 200, 3, 40], [100, 300, 20, 60], 4, 2, seed=10, wide=wide)
    want, ref = c.run(), c.reference()[0]
    kw = {}
    if case == "page":
        c.table[1, 2] = c.kc.shape[0]
        hurt = [1]
    elif case == "length":
        c.tlens[2] = -1
        hurt = [2]
    elif case == "long":
        c.tlens[1] = c.table.shape[1] * c.page + 1
        hurt = [1]
    elif case == "offset":
        c.tstart[2] = 300  # (behind the rows, and behind the next)
        hurt = [1, 2]
    elif case == "behind":
        c.tstart[4] += 1
        hurt = [3]
    else:
        kw = dict(max_new=100)
        hurt = [1]
    out = torch.zeros_like(want)
    from transformer_encoder_gb300 import chunk_attention
    chunk_attention(c.q, c.kc, c.vc, c.table, c.tlens, seq_start=c.tstart, out=out, **{"max_new": 200, **kw})
    with pytest.raises(WencError, match="out of range") as e:
        sync_status()
    assert e.value.status == 1
    # (not bit by bit: where long rows are cut into pieces depends on the whole call; within the bound of the rounding)
    for s in range(4):
        if s not in hurt:
            rows = slice(int(c.start[s]), int(c.start[s + 1]))
            limit = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -19
            assert float((out[rows].double() - ref[rows]).norm()) <= limit * float(ref[rows].norm()), s


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", [False, True])
def test_strided_tensors(dtype, wide):
    import torch
    c = Case(dtype, [1, 60, 300], [100, 3, 500], 6, 2, page=24, strided=True, odd_pages=True, seed=11, wide=wide)
    around = torch.full((c.q.shape[0], 10, 64), 5.0, device="cuda", dtype=c.dt)
    out = around[:, 2:8]
    table = torch.full((3, c.table.shape[1] + 5), -9, dtype=torch.int32, device="cuda")
    table[:, 2:2 + c.table.shape[1]] = c.table
    c.table = table[:, 2:2 + c.table.shape[1]]
    c.check(c.run(out=out))
    assert (around[:, :2] == 5).all() and (around[:, 8:] == 5).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_offsets_past_32_bits(dtype):
    """Pages in the last of more than 2^32 elements' worth of cache."""
    import torch
    Hkv, page, es = 4, 64, 2 if dtype == "bf16" else 4
    n_pages = (1 << 32) // (page * Hkv * 64) + 64
    c = Case(dtype, [1, 150], [600, 200], 8, Hkv, page=page, seed=12)
    big_k, big_v = (torch.empty(n_pages, page, Hkv, 64, dtype=c.dt, device="cuda") for _ in range(2))
    total = c.kc.shape[0]
    big_k[-total:], big_v[-total:] = c.kc, c.vc
    want = c.run()
    c.kc, c.vc = big_k, big_v
    c.table = torch.where((c.table >= 0) & (c.table < total), c.table + n_pages - total, torch.full_like(c.table, -1))
    assert torch.equal(c.run(), want)
    assert es * big_k.numel() > 1 << 32


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wide", [False, True])
def test_streams_workspaces_and_graphs(dtype, wide):
    """On a stream of its own, with a given workspace, captured and replayed with other lengths."""
    import torch
    from transformer_encoder_gb300 import chunk_attention, sync_status
    c = Case(dtype, [1, 200, 3, 40], [100, 300, 20, 600], 4, 2, seed=13, wide=wide)
    want = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    room = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    args = (c.q, c.kc, c.vc, c.table, c.tlens)
    kw = dict(seq_start=c.tstart, max_new=200, out=out, workspace=room)
    chunk_attention(*args, **kw, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chunk_attention(*args, **kw)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    c.tlens -= 20  # shorter caches: the graph follows
    graph.replay()
    again = chunk_attention(*args, seq_start=c.tstart, max_new=200)
    torch.cuda.synchronize()
    assert torch.equal(out, again) and not torch.equal(again, want)
    sync_status()


def test_what_the_binding_refuses():
    import torch
    from transformer_encoder_gb300 import chunk_attention
    c = Case("bf16", [1, 2], [10, 20], 4, 2)
    args = [c.q, c.kc, c.vc, c.table, c.tlens]
    for i, bad, err in ((0, c.q.half(), TypeError), (0, c.q[:, :3], Exception), (0, c.q.view(1, 3, 4, 64), ValueError),
                        (1, c.kc.float(), TypeError), (2, c.vc[:, :, :1], ValueError), (3, c.table.long(), TypeError),
                        (3, c.table[:1], ValueError), (4, c.tlens.long(), TypeError), (0, c.q.cpu(), TypeError),
                        (4, c.tlens.cpu(), TypeError)):
        with pytest.raises(err):
            chunk_attention(*[bad if j == i else a for j, a in enumerate(args)], seq_start=c.tstart)
    for kw in (dict(seq_start=c.tstart[:2]), dict(window=0), dict(window=4, sinks=-1), dict(sinks=3), dict(out=c.q.float()),
               dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda")[::2]), dict(max_new=0)):
        with pytest.raises(Exception):
            chunk_attention(*args, **{"seq_start": c.tstart, **kw})
    assert chunk_attention(c.q[:0], *args[1:], seq_start=torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 4, 64)


def test_tokens_of_no_sequence_are_refused():
    import torch
    from transformer_encoder_gb300 import chunk_attention
    c = Case("bf16", [1, 2], [10, 20], 4, 2)
    none = dict(block_table=c.table[:0], lens=c.tlens[:0])
    with pytest.raises(ValueError, match="no sequence"):
        chunk_attention(c.q, c.kc, c.vc, **none)
    start = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert (chunk_attention(c.q, c.kc, c.vc, **none, seq_start=start) == 0).all()  # (all of it padding)


@pytest.mark.parametrize("dtype", DTYPES)
def test_queries_and_results_side_by_side(dtype):
    """Results into other columns of the rows that the queries come from; into the queries' own they are refused."""
    import torch
    c = Case(dtype, [1, 90, 4], [200, 30, 9], 4, 2, seed=18, wide=True)
    rows = torch.full((c.q.shape[0], 12, 64), 3.0, device="cuda", dtype=c.dt)
    rows[:, 1:5] = c.q
    want = c.run()
    c.q = rows[:, 1:5]
    assert torch.equal(c.run(out=rows[:, 6:10]), want)
    assert (rows[:, 0] == 3).all() and (rows[:, 5] == 3).all() and (rows[:, 10:] == 3).all()
    with pytest.raises(Exception, match="apart"):
        c.run(out=rows[:, 4:8])
