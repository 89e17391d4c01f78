"""wenc_prefix_attention against its float64 definition, at the sizes and lengths where it can go wrong.

Bounds, from the arithmetic. Let A = max_j sum_i |q_i k_ij| of the row and n the keys it sees.
bf16: products of bf16 are exact in fp32; 64 of them accumulate with at most 64 roundings of 2^-23
relative to A each (the tensor core may truncate), so a score is off by d = scale * A * 64 * 2^-23,
plus two roundings of the exponent's argument (at most 2 * 128 * 2^-24 = 2^-16 in log2 units: inputs
are scaled so that |argument| < 128) and 2^-21 for exp2: p is off by e = 1.1 d + 2^-16 + 2^-21
relative, numerator and denominator both. P enters the product as two bf16 parts: 2^-16 more in the
numerator. Sums over n keys: n * 2^-23 each. Output rounding: 2^-8 (half a step of bf16).
  |err| <= 2^-8 |o| + (2 e + 2^-16 + 2 n 2^-23) sum_j p_j |v_j|
bf16, more than 64 rows per key head behind a prefix: where that is the tcgen05 form, P enters as one bf16
number, 2^-8 instead of 2^-16 in the numerator.
fp32: every operand is two TF32 parts that miss it by less than 2^-22 (11 bits rounded, 11 more of the rest cut
off), the product of the small parts (2^-11 each) is dropped: 3 * 2^-22 a product, and three times as many
accumulations; output 2^-24:
  d = scale * A * (3 * 2^-22 + 192 * 2^-23), and in the numerator 3 * 2^-22 + 4 n 2^-23.
"""
import numpy as np
import pytest

import synth
from oracle import decode

pytestmark = pytest.mark.gpu


def _dev(a, dtype):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def _i32(a):
    import torch
    return torch.tensor(list(a), dtype=torch.int32, device="cuda")


class Case:
    """Host values and device tensors of one problem. Everything behind a length holds NaN."""

    def __init__(self, dtype, sizes, q_len, H, Hkv, pre, suf, page=16, seed=0, uneven=False, prefix_max=None, extra=0,
                 pad_pages=0, strided=False):
        import torch
        r = np.random.default_rng(seed)
        rnd = (lambda *s: synth.round_to_bf16(r.standard_normal(s).astype(np.float32))) if dtype == "bf16" else (
            lambda *s: r.standard_normal(s).astype(np.float32))
        self.dtype, self.q_len, self.H, self.Hkv = dtype, q_len, H, Hkv
        n = sum(sizes) + extra  # `extra` sequences behind the last group
        self.n, self.n_in = n, sum(sizes)
        self.groups = [g for g, s in enumerate(sizes) for _ in range(s)]
        self.q = rnd(n, q_len, H, 64)
        self.kw = {}
        self.prefixes = [(np.zeros((0, Hkv, 64)), np.zeros((0, Hkv, 64)))] * len(sizes)
        if pre is not None:
            T = prefix_max or max(max(pre), 1)
            kp, vp = np.full((len(sizes), T, Hkv, 64), np.nan, np.float32), np.full((len(sizes), T, Hkv, 64), np.nan, np.float32)
            self.prefixes = []
            for g, m in enumerate(pre):
                k, v = rnd(m, Hkv, 64), rnd(m, Hkv, 64)
                kp[g, :m], vp[g, :m] = k, v
                self.prefixes.append((k.astype(np.float64), v.astype(np.float64)))
            self.kw.update(k_prefix=_dev(kp, dtype), v_prefix=_dev(vp, dtype), prefix_lens=_i32(pre))
            if uneven:
                self.kw.update(group_start=_i32(np.cumsum([0] + list(sizes))), max_group=max(sizes))
        self.owns = [(np.zeros((0, Hkv, 64)), np.zeros((0, Hkv, 64)))] * n
        if suf is not None:
            need = [-(-m // page) for m in suf]
            total, width = max(1, sum(need)) + pad_pages, max(1, max(need)) + 1
            order = r.permutation(total)
            kc, vc = np.full((total, page, Hkv, 64), np.nan, np.float32), np.full((total, page, Hkv, 64), np.nan, np.float32)
            table = np.full((n, width), -1, np.int32)
            self.owns, at = [], 0
            for s, m in enumerate(suf):
                k, v = rnd(m, Hkv, 64), rnd(m, Hkv, 64)
                table[s, :need[s]] = order[at:at + need[s]]
                for j in range(m):
                    kc[table[s, j // page], j % page] = k[j]
                    vc[table[s, j // page], j % page] = v[j]
                at += need[s]
                self.owns.append((k.astype(np.float64), v.astype(np.float64)))
            self.kw.update(k_pages=_dev(kc, dtype), v_pages=_dev(vc, dtype), lens=_i32(suf),
                           block_table=torch.from_numpy(table).cuda())
        if strided:  # queries inside wider rows
            wide = np.full((n, q_len, H + 3, 64), np.nan, np.float32)
            wide[:, :, 1:1 + H] = self.q
            self.tq = _dev(wide, dtype)[:, :, 1:1 + H]
        else:
            self.tq = _dev(self.q, dtype)

    def run(self, **kw):
        from transformer_encoder_gb300 import prefix_attention, sync_status
        out = prefix_attention(self.tq, **self.kw, **kw)
        sync_status()
        return out

    def check(self, out, scale=0.125, what=""):
        import torch
        got = out.to(torch.float64).cpu().numpy()[:self.n_in]
        ref, absv, A = decode.prefix_attention(self.q[:self.n_in].astype(np.float64), self.prefixes, self.owns,
                                               self.groups, scale)
        keys = max(p[0].shape[0] for p in self.prefixes) + max(o[0].shape[0] for o in self.owns)
        A = A[..., None] * abs(scale)
        assert (1.4427 * A < 128).all()
        e = 2.0 ** -16 + 2.0 ** -21
        one_part = bool(self.prefixes[0][0].shape[0] or len(self.prefixes) > 1) and "k_prefix" in self.kw and (
            max(self.groups.count(g) for g in set(self.groups)) * self.q_len * self.H > 64 * self.Hkv)
        if self.dtype == "bf16":
            e = e + 1.1 * A * 64 * 2.0 ** -23
            bound = 2.0 ** -8 * np.abs(ref) + (2 * e + (2.0 ** -8 if one_part else 2.0 ** -16) + 2 * keys * 2.0 ** -23) * absv
        else:
            e = e + 1.1 * A * (3 * 2.0 ** -22 + 192 * 2.0 ** -23)
            bound = 2.0 ** -24 * np.abs(ref) + (2 * e + 3 * 2.0 ** -22 + 4 * keys * 2.0 ** -23) * absv
        assert np.isfinite(got).all(), what
        err = np.abs(got - ref)
        assert (err <= bound + 1e-30).all(), f"{what}: {float((err / (bound + 1e-30)).max()):.2f} x the bound"
        if np.linalg.norm(ref) > 0:  # what a systematic mistake under the elementwise bound would show
            # (bf16: elementwise half steps; fp32: the score errors of a row of 64, some 2^-19)
            assert np.linalg.norm(got - ref) <= (2.0 ** -8 * (1.5 if one_part else 1) if self.dtype == "bf16" else 2.0 ** -19) * np.linalg.norm(ref), what


DTYPES = ["bf16", "f32"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("keys", [1, 7, 16, 33, 64, 127, 128, 129, 300, 1500])
def test_prefix_only_lengths(dtype, keys):
    """One beam group over prefixes from one key to a window's 1500."""
    c = Case(dtype, [5], 1, 6, 6, [keys], None, seed=keys)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("own", [1, 2, 15, 16, 17, 63, 128, 257])
@pytest.mark.parametrize("page", [1, 3, 16, 64])
def test_own_keys_only(dtype, own, page):
    """No prefix: pages of odd sizes, lengths that end inside a page and a tile, an empty sequence."""
    c = Case(dtype, [1, 1, 1], 1, 4, 2, None, [own, 0, max(1, own // 2)], page=page, seed=own * 7 + page)
    out = c.run()
    c.check(out)
    assert (out[1] == 0).all()  # sees nothing


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 6), (20, 4), (5, 1), (16, 2)])
@pytest.mark.parametrize("q_len", [1, 3, 8])
def test_head_layouts_and_draft_tokens(dtype, H, Hkv, q_len):
    """Shared key heads and several causal tokens; own lengths shorter than the tokens among them."""
    c = Case(dtype, [2, 2], q_len, H, Hkv, [40, 0], [q_len, 50, max(0, q_len - 2), 0], page=8, seed=H * 10 + q_len)
    out = c.run()
    c.check(out)
    assert (out[3] == 0).all()  # group without prefix, no own keys


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", [[1, 4, 2], [3, 0, 5, 1], [17, 2], [70], [130, 1]])
def test_uneven_groups(dtype, sizes):
    """Groups of any size (an empty one among them), rows past one and several row tiles."""
    r = np.random.default_rng(sum(sizes))
    pre = [int(r.integers(0, 200)) for _ in sizes]
    c = Case(dtype, sizes, 1, 4, 2, pre, [int(r.integers(0, 40)) for _ in range(sum(sizes))], uneven=True, seed=1,
             prefix_max=220)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hkv,pre", [(3, 1, None), (2, 2, [70, 0]), (40, 20, None), (40, 20, [300, 65])])
def test_long_drafts(dtype, H, Hkv, pre):
    """Many new tokens a sequence: rows of one sequence over many tiles, causal among its newest keys; own keys fewer
    than, as many as, and more than the tokens."""
    sizes = [3, 2] if pre else [1] * 5
    c = Case(dtype, sizes, 130, H, Hkv, pre, [200, 130, 64, 0, 131], page=24, uneven=pre is not None, seed=26)
    assert _joins(c) == (H == 40)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [1, 3, 5, 1000])
def test_page_sizes(dtype, page):
    c = Case(dtype, [2, 3], 2, 4, 2, [20, 33], [17, 100, 2, 64, 31], page=page, uneven=True, seed=27)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_no_group_stay(dtype):
    """Sequences behind the last group keep their rows of the output."""
    import torch
    for suf in (None, [3, 9, 1, 5, 6, 7]):
        c = Case(dtype, [2, 2], 2, 2, 2, [9, 30], suf, uneven=True, extra=2, seed=3)
        out = torch.full_like(c.tq, 7.0)
        got = c.run(out=out)
        assert got is out
        c.check(out)
        assert (out[4:] == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_inputs(dtype):
    """Queries inside wider rows, output likewise, K and V prefix interleaved, pages of one pool."""
    import torch
    c = Case(dtype, [3], 2, 4, 4, [50], [10, 20, 30], strided=True, seed=4)
    k, v = c.kw["k_prefix"], c.kw["v_prefix"]
    both = torch.stack([k, v], dim=2)  # [G, T, 2, H, 64]
    c.kw["k_prefix"], c.kw["v_prefix"] = both[:, :, 0], both[:, :, 1]
    pool = torch.stack([c.kw["k_pages"], c.kw["v_pages"]], dim=1)  # [pages, 2, page, H, 64]
    c.kw["k_pages"], c.kw["v_pages"] = pool[:, 0], pool[:, 1]
    wide = torch.zeros(3, 2, 6, 64, dtype=c.tq.dtype, device="cuda")
    c.check(c.run(out=wide[:, :, :4]))
    assert (wide[:, :, 4:] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [0.125, 1.0 / 3, -0.2, 0.0])
def test_scales(dtype, scale):
    c = Case(dtype, [2], 1, 2, 2, [70], [9, 12], seed=5)
    c.check(c.run(scale=scale), scale)


@pytest.mark.parametrize("dtype", DTYPES)
def test_far_apart_scores_and_extreme_values(dtype):
    """A key that takes all the weight, in the prefix or among the own keys; and keys whose scores
    lie so far below that they vanish."""
    import torch
    c = Case(dtype, [2], 1, 2, 2, [40], [20, 20], seed=6)
    q, kp, kc = c.tq, c.kw["k_prefix"], c.kw["k_pages"]
    kp[0, 17] = q[0, 0] * 8  # dominates sequence 0
    out = c.run()
    torch.cuda.synchronize()
    want = c.kw["v_prefix"][0, 17]
    assert torch.allclose(out[0, 0].float(), want.float(), rtol=2.0 ** -7, atol=1e-4)
    kp[0, 17] = q[0, 0] * -8
    page, slot = int(c.kw["block_table"][0, 0]), 3
    kc[page, slot] = q[0, 0] * 8
    out = c.run()
    assert torch.allclose(out[0, 0].float(), c.kw["v_pages"][page, slot].float(), rtol=2.0 ** -7, atol=1e-4)


def test_many_rows_behind_a_long_prompt():
    """More rows than a row tile and keys over many splits, key heads shared by five query heads."""
    c = Case("bf16", [40], 1, 10, 2, [2050], [int(x) for x in np.random.default_rng(0).integers(1, 90, 40)], page=64,
             seed=7)
    c.check(c.run())


def _joins(c):
    """Whether the case runs in the form that joins partial results (it alone needs a workspace)."""
    import torch
    from transformer_encoder_gb300 import WencError, prefix_attention
    try:
        prefix_attention(c.tq, **c.kw, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    except WencError as e:
        return "workspace" in str(e)
    return False


@pytest.mark.parametrize("H,Hkv,q_len,sizes,pre", [
    (32, 32, 1, [160], [1]), (32, 32, 1, [165], [129]), (96, 32, 1, [60, 5], [257, 0]), (48, 16, 4, [30, 1, 25], [128, 700, 5]),
    (80, 16, 1, [70], [900]), (40, 1, 1, [130, 2], [300, 64]), (128, 1, 1, [45], [200]), (4, 4, 7, [40, 180], [500, 127]),
    (96, 32, 1, [70], [0]), (1, 1, 1, [2500], [1700])])
@pytest.mark.parametrize("own", [False, True])
def test_many_rows(H, Hkv, q_len, sizes, pre, own):
    """The tcgen05 form: grouped heads that do and do not divide a tile's 128 rows, several row tiles,
    groups without rows or keys, lengths around a key tile, with and without own keys; NaN behind every
    length."""
    r = np.random.default_rng(sum(sizes) + H)
    suf = [int(r.integers(0, 20)) for _ in range(sum(sizes))] if own else None
    c = Case("bf16", sizes, q_len, H, Hkv, pre, suf, page=8, uneven=len(sizes) > 1, seed=H + q_len, prefix_max=max(pre) + 37,
             strided=own)
    assert _joins(c)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hkv,q_len,sizes,pre", [
    (2, 2, 1, [65], [1]), (2, 2, 1, [300], [129]), (6, 2, 1, [90, 5], [257, 0]), (6, 2, 4, [30, 1, 25], [128, 700, 5]),
    (5, 1, 1, [51], [1500]), (40, 1, 1, [7, 2], [300, 64]), (128, 1, 1, [3], [200]), (4, 4, 7, [10, 40], [1000, 127])])
def test_many_rows_of_little_work(dtype, H, Hkv, q_len, sizes, pre):
    """More than 64 rows in the one-launch form (fp32: where the work is less than 3 * 2^18 pairs of a row and a
    key): several row tiles per group, each over the whole prefix."""
    r = np.random.default_rng(sum(sizes) + H)
    c = Case(dtype, sizes, q_len, H, Hkv, pre, [int(r.integers(0, 20)) for _ in range(sum(sizes))], page=8,
             uneven=len(sizes) > 1, seed=H + q_len, prefix_max=max(pre) + 37, strided=True)
    pairs = len(sizes) * H * q_len * max(sizes) * (max(pre) + 37)
    assert _joins(c) == (dtype == "f32" and pairs > 3 << 18)
    c.check(c.run())


@pytest.mark.parametrize("H,Hkv,q_len,sizes,pre", [
    (32, 32, 1, [245], [129]), (48, 16, 4, [10, 1, 25], [128, 300, 5]), (96, 32, 1, [60, 5], [257, 0]), (80, 16, 1, [70], [900]),
    (40, 1, 1, [130, 2], [300, 64]), (128, 1, 1, [45], [200]), (130, 1, 1, [50], [150]), (4, 4, 7, [40, 180], [500, 127]),
    (1, 1, 1, [2500], [1700]), (8, 8, 1, [1200], [1]), (8, 8, 1, [1200], [63]), (8, 8, 1, [1200], [64]), (8, 8, 1, [1200], [65]),
    (16, 16, 1, [70, 70, 69, 3], [450, 449, 192, 1])])
@pytest.mark.parametrize("own", [False, True])
def test_many_rows_f32(H, Hkv, q_len, sizes, pre, own):
    """The form that joins partial results, fp32: on tcgen05 up to 128 query heads per key head."""
    r = np.random.default_rng(sum(sizes) + H)
    suf = [int(r.integers(0, 20)) for _ in range(sum(sizes))] if own else None
    c = Case("f32", sizes, q_len, H, Hkv, pre, suf, page=8, uneven=len(sizes) > 1, seed=H + q_len, prefix_max=max(pre) + 37,
             strided=own)
    assert _joins(c)
    c.check(c.run())


def test_many_heads_per_key_head_bf16():
    """More query heads per key head than a tcgen05 row tile holds."""
    c = Case("bf16", [300], 1, 130, 1, [300], None, seed=25)
    assert _joins(c)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [0.125, 0.3, -0.2, 0.0])
def test_many_rows_scales(dtype, scale):
    c = Case(dtype, [160], 1, 32, 32, [300], [int(x) for x in np.random.default_rng(0).integers(0, 9, 160)], seed=15)
    assert _joins(c)
    c.check(c.run(scale=scale), scale)


def test_many_rows_on_another_stream_and_in_two_graphs():
    """The forms that need a workspace: on a given stream, and as two captured graphs replayed at once, each
    with the workspace of its own capture."""
    import torch
    from transformer_encoder_gb300 import prefix_attention
    cases = [Case("bf16", [170], 1, 32, 32, [700], [30] * 170, seed=s) for s in (17, 18)]
    cases.append(Case("f32", [245], 1, 32, 32, [100], [30] * 245, seed=19))
    assert all(_joins(c) for c in cases)
    want = [c.run() for c in cases]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        out = prefix_attention(c.tq, **c.kw, stream=s)
        s.synchronize()
        assert torch.equal(out, w)
    graphs, outs = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(prefix_attention(c.tq, **c.kw))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [3, 70, 3700])
def test_nan_queries_and_keys_reach_their_rows_alone(dtype, size):
    """A NaN query, and a NaN among a sequence's visible own keys, make those rows NaN and no others,
    in the one-launch form and in the one that joins partial results."""
    import torch
    from transformer_encoder_gb300 import prefix_attention, sync_status
    c = Case(dtype, [size], 1, 2, 2, [50], [9] * size, seed=20)
    assert _joins(c) == (size == 3700)
    want = c.run()
    q = c.tq.clone()
    q[1, 0, 0] = float("nan")
    kc = c.kw["k_pages"].clone()
    kc[int(c.kw["block_table"][2, 0]), 4, 1] = torch.zeros(1, device="cuda").log().neg().sub(float("inf"))  # the GPU's NaN
    out = prefix_attention(q, **{**c.kw, "k_pages": kc})
    sync_status()
    bad = torch.zeros(size, 1, 2, dtype=torch.bool, device="cuda")
    bad[1, 0, 0] = bad[2, 0, 1] = True
    assert torch.isnan(out[bad]).all()
    assert torch.equal(out[~bad], want[~bad])


def test_many_rows_of_no_group_stay():
    import torch
    c = Case("bf16", [80, 66], 1, 32, 32, [90, 130], None, uneven=True, extra=3, seed=16)
    assert _joins(c)
    out = torch.full_like(c.tq, 7.0)
    c.check(c.run(out=out))
    assert (out[146:] == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [2, 70, 3700])
def test_padding_sequences_may_hold_anything(dtype, size):
    """Lengths and page numbers of sequences behind the last group are not looked at, in any form."""
    import torch
    c = Case(dtype, [size, 1], 1, 2, 2, [50, 30], [9] * (size + 4), uneven=True, extra=3, seed=23)
    assert _joins(c) == (size == 3700)
    c.kw["lens"][-3:] = _i32([-5, 10 ** 9, 3])
    c.kw["block_table"][-3:] = -7
    out = torch.full_like(c.tq, 7.0)
    c.check(c.run(out=out))
    assert (out[-3:] == 7.0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [3, 70, 3700])
def test_scores_below_every_number_weigh_nothing(dtype, size):
    """Finite queries and keys whose products pass fp32's range: such scores are -inf, alone in a tile, in
    a share of the prefix, and before and behind keys that count."""
    import torch
    c = Case(dtype, [size], 1, 2, 2, [700], None, seed=24)
    c.q[..., 0] = 16.0
    c.tq = _dev(c.q, dtype)
    c.kw["k_prefix"][0, :256, :, 0] = -3e38
    c.kw["k_prefix"][0, 400:, :, 0] = -3e38
    k, v = c.prefixes[0]
    c.prefixes = [(k[256:400], v[256:400])]
    c.check(c.run())
    c.kw["prefix_lens"] = _i32([200])  # no other keys: no weight is a number
    assert not torch.isinf(c.run()).any()


def test_large_prefix_group_f32_draft_rows():
    c = Case("f32", [9, 9], 3, 4, 2, [700, 651], [int(x) for x in np.random.default_rng(0).integers(0, 60, 18)], page=24,
             seed=8)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
def test_replayed_graph_follows_the_lengths(dtype):
    """One captured step, replayed with other lengths, queries and tables."""
    import torch
    from transformer_encoder_gb300 import prefix_attention, sync_status
    a = Case(dtype, [2, 2], 1, 4, 4, [60, 33], [5, 30, 17, 48], seed=9, prefix_max=64)
    b = Case(dtype, [2, 2], 1, 4, 4, [1, 64], [48, 2, 0, 31], seed=10, prefix_max=64)
    width = max(a.kw["block_table"].shape[1], b.kw["block_table"].shape[1])
    pages = max(a.kw["k_pages"].shape[0], b.kw["k_pages"].shape[0])
    live = {}
    for name, t in a.kw.items():
        shape = list(t.shape)
        if name == "block_table":
            shape[1] = width
        if name.endswith("_pages"):
            shape[0] = pages
        live[name] = torch.full(shape, -1 if t.dtype == torch.int32 else float("nan"), dtype=t.dtype, device="cuda")
    q = torch.empty_like(a.tq)

    def fill(c):
        q.copy_(c.tq)
        for name, t in c.kw.items():
            live[name].fill_(-1 if t.dtype == torch.int32 else float("nan"))
            live[name][tuple(slice(0, m) for m in t.shape)].copy_(t)

    fill(a)
    prefix_attention(q, **live)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = prefix_attention(q, **live)
    for c in (b, a, b):
        fill(c)
        out.fill_(3.0)
        g.replay()
        sync_status()
        c.check(out)


def test_two_streams_at_once_and_given_workspace():
    """Calls on two streams, each with a workspace of its own, give what they give alone; a repeated
    call gives the same bits whatever the workspace held."""
    import torch
    from transformer_encoder_gb300 import prefix_attention
    cases = [Case("bf16", [5, 5], 1, 6, 6, [900, 700], [20] * 10, seed=s) for s in (11, 12)]
    alone = [c.run() for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for c, s, o in zip(cases, streams, outs):
            with torch.cuda.stream(s):
                o.append(prefix_attention(c.tq, **c.kw))
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        for x in o:
            assert torch.equal(a, x)
    ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(cases[0].run(workspace=ws, stream=s), alone[0])


def test_offsets_past_32_bits():
    """Keys more than 2^32 bytes from the start of the prefix and of the pages."""
    import torch
    from transformer_encoder_gb300 import prefix_attention, sync_status
    H = 4
    T = (1 << 32) // (H * 64 * 2) + 64  # prefix of 2^32 bytes and some
    big = torch.zeros(1, T, H, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    big[:, -64:] = torch.randn(1, 64, H, 64, generator=g, device="cuda").to(torch.bfloat16)
    q = torch.randn(1, 1, H, 64, generator=g, device="cuda").to(torch.bfloat16) * 4
    out = prefix_attention(q, big, big)
    sync_status()
    k = big[0, -64:].double()
    z = (k * q[0, 0].double()).sum(2) / 8
    m = z.max(0).values.clamp(min=0)
    p = torch.exp(z - m)
    den = p.sum(0) + (T - 64) * torch.exp(-m)  # the zero keys score 0 and add nothing to the numerator
    ref = (p.unsqueeze(2) * k).sum(0) / den.unsqueeze(1)
    assert (out[0, 0].double() - ref).abs().max() <= 2.0 ** -7 * ref.abs().max()
    pages = big.view(-1, 64, H, 64)
    table = torch.tensor([[pages.shape[0] - 1]], dtype=torch.int32, device="cuda")
    out = prefix_attention(q, k_pages=pages, v_pages=pages, block_table=table, lens=_i32([64]))
    sync_status()
    ref = (torch.softmax(z, 0).unsqueeze(2) * k).sum(0)
    assert (out[0, 0].double() - ref).abs().max() <= 2.0 ** -7 * ref.abs().max()


@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length", "prefix length", "offsets", "group"])
def test_bad_device_data_is_reported(what):
    """Lengths, offsets and page numbers out of range: reported, nothing out of range accessed, and
    the next call is clean again."""
    _bad_device_data(Case("bf16", [2, 2], 1, 2, 2, [20, 30], [10, 20, 18, 17], seed=13, uneven=True, prefix_max=32), what)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length", "prefix length", "offsets", "group"])
def test_bad_device_data_is_reported_by_many_rows(dtype, what):
    c = Case(dtype, [130, 130], 1, 32, 32, [20, 30], [17] * 260, seed=13, uneven=True, prefix_max=32)
    assert _joins(c)
    _bad_device_data(c, what)


def _bad_device_data(c, what):
    import torch
    from transformer_encoder_gb300 import WencError, prefix_attention, sync_status
    kw = {k: v.clone() if torch.is_tensor(v) else v for k, v in c.kw.items()}
    if what == "page":
        kw["block_table"][1, 0] = kw["k_pages"].shape[0]
    if what == "negative page":
        kw["block_table"][1, 0] = -1
    if what == "length":
        kw["lens"][2] = kw["block_table"].shape[1] * 16 + 1
    if what == "negative length":
        kw["lens"][2] = -1
    if what == "prefix length":
        kw["prefix_lens"][0] = 33
    if what == "offsets":
        kw["group_start"][1] = 1 << 20
    if what == "group":
        kw["group_start"][1] = kw["max_group"] + 1
    prefix_attention(c.tq, **kw)
    with pytest.raises(WencError, match="out of range") as e:
        sync_status()
    assert e.value.status == 1
    c.check(c.run())
