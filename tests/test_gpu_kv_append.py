"""wenc_kv_append against its float64 definition.

Bounds, from the arithmetic: the angle is good to 2^-31 of a turn before the fp32 sine and cosine
(2^-21 absolute is more than their error and that of the angle together), the two products and their
sum are rounded in fp32 (3 * 2^-24), the result once to the stored type (half a step: 2^-8 for bf16,
2^-24 for fp32): |err| <= u |y| + (2^-21 + 3 * 2^-24) (|x_a| + |x_b|). What does not turn is copied bit
for bit.
"""
import numpy as np
import pytest

import synth
from oracle import decode

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _torch_dtype(dtype):
    import torch
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _inv_freq(rot):
    return np.array([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], np.float32)


class Case:
    def __init__(self, dtype, new, past, H, Hkv, rot, interleaved=False, page=16, pad=0, positions=None, seed=0, with_q=True,
                 inv_freq=None):
        import torch
        r = np.random.default_rng(seed)
        n = sum(new) + pad
        self.n, self.rows, self.H, self.Hkv, self.dtype = sum(new), n, H, Hkv, dtype
        x = r.standard_normal((n, H + 2 * Hkv, 64)).astype(np.float32)
        if dtype == "bf16":
            x = synth.round_to_bf16(x)
        self.x = x.astype(np.float64)
        self.fused = torch.from_numpy(x).cuda().to(_torch_dtype(dtype))
        self.q, self.k, self.v = self.fused[:, :H], self.fused[:, H:H + Hkv], self.fused[:, H + Hkv:]
        self.lens = [p + m for p, m in zip(past, new)]
        need = [-(-m // page) for m in self.lens]
        total = sum(need) + 2
        order = r.permutation(total)
        self.table = np.full((len(new), max(1, max(need)) + 1), -1, np.int32)
        at = 0
        for s, m in enumerate(need):
            self.table[s, :m] = order[at:at + m]
            at += m
        self.page, self.interleaved = page, interleaved
        self.pos = np.concatenate([np.arange(v - m, v) for m, v in zip(new, self.lens)] + [np.zeros(0, int)]).astype(np.int64)
        self.seq = np.repeat(np.arange(len(new)), new)
        self.kc = torch.full((total, page, Hkv, 64), 5.0, dtype=_torch_dtype(dtype), device="cuda")
        self.vc = torch.full((total, page, Hkv, 64), 6.0, dtype=_torch_dtype(dtype), device="cuda")
        self.kw = dict(seq_start=torch.tensor(np.cumsum([0] + list(new)), dtype=torch.int32, device="cuda"))
        self.turn = self.pos
        if positions is not None:
            self.turn = np.asarray(positions[:self.n], np.int64)
            self.kw["positions"] = torch.tensor(np.asarray(positions), dtype=torch.int32, device="cuda")
        self.freq = None
        if rot:
            self.freq = _inv_freq(rot) if inv_freq is None else np.asarray(inv_freq, np.float32)
            self.kw.update(inv_freq=torch.from_numpy(self.freq).cuda(), interleaved=interleaved)
        if with_q:
            self.kw["q"] = self.q

    def run(self, **kw):
        import torch
        from transformer_encoder_gb300 import kv_append, sync_status
        out = kv_append(self.k, self.v, self.kc, self.vc, torch.from_numpy(self.table).cuda(),
                        torch.tensor(self.lens, dtype=torch.int32, device="cuda"), **{**self.kw, **kw})
        sync_status()
        return out

    def check(self, q_out=None):
        H, Hkv, n = self.H, self.Hkv, self.n
        ids, slots = self.table[self.seq, self.pos // self.page], self.pos % self.page

        def near(got, x, what):
            if self.freq is None:
                assert np.array_equal(got, x), what
                return
            y, mag = decode.rotate(x, self.turn, self.freq, self.interleaved)
            bound = U[self.dtype] * np.abs(y) + (2.0 ** -21 + 3 * 2.0 ** -24) * mag
            still = 2 * len(self.freq)
            assert np.array_equal(got[:, :, still:], x[:, :, still:]), what
            assert (np.abs(got - y) <= bound).all(), what

        host = lambda t: t.double().cpu().numpy()
        kc, vc = host(self.kc), host(self.vc)
        near(kc[ids, slots], self.x[:n, H:H + Hkv], "keys")
        assert np.array_equal(vc[ids, slots], self.x[:n, H + Hkv:])
        rest = np.ones(kc.shape[:2], bool)  # every other slot as it was
        rest[ids, slots] = False
        assert (kc[rest] == 5.0).all() and (vc[rest] == 6.0).all()
        if q_out is not None:
            near(host(q_out)[:n], self.x[:n, :H], "queries")


DTYPES = ["bf16", "f32"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32, 48, 64])
def test_rotations(dtype, interleaved, rot):
    c = Case(dtype, [3, 1, 5], [7, 0, 30], 4, 2, rot, interleaved, seed=rot)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 6), (20, 4), (5, 1), (20, 20)])
@pytest.mark.parametrize("new", [[1], [0, 1, 0], [2, 0, 3, 1, 1], [40, 33]])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_layouts(dtype, H, Hkv, new, page):
    """Head layouts, empty sequences at the start, middle and end, pages of odd sizes."""
    c = Case(dtype, new, [(5 * i + 3) % 50 for i in range(len(new))], H, Hkv, 64, page=page, seed=H)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n_seqs", [31, 32, 33, 500, 1100])
def test_many_sequences(dtype, n_seqs):
    """The search for a token's sequence over one, two and three steps of 32, with empty sequences."""
    r = np.random.default_rng(n_seqs)
    new = [int(r.integers(0, 4)) for _ in range(n_seqs)]
    c = Case(dtype, new, [int(r.integers(0, 9)) for _ in range(n_seqs)], 2, 1, 32, page=8, pad=9, seed=n_seqs)
    c.check(c.run())


def test_long_chunks():
    """Enough tokens that a warp takes several in a row, across sequence ends."""
    c = Case("bf16", [9001, 0, 1, 12007, 333], [0, 5, 2, 100, 0], 2, 2, 64, page=64, pad=50, seed=2)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("far", [0, 4095, 1 << 20, (1 << 31) - 64, -1000])
def test_far_positions(dtype, far):
    """The angle of a position near 2^31 is as good as that of a near one; positions may be negative."""
    c = Case(dtype, [20, 13], [0, 4], 2, 2, 64, positions=[far + i for i in range(33)], seed=3)
    c.check(c.run())


def test_other_frequencies():
    """Frequencies beyond a turn per position, negative, zero and tiny ones."""
    f = [7.5, -0.3, 0.0, 1e-30, 100.0, 6.2831855, 3.1415927, 1e-8]
    c = Case("f32", [50], [1000], 1, 1, 16, inv_freq=f, seed=4)
    c.check(c.run())


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 64, -(1 << 31)])
def test_negative_frequencies_at_far_positions(far):
    """A negative frequency turns back by exactly what the positive one turns forward."""
    f = np.concatenate([-_inv_freq(16), [-0.3, -1e-6, -7.5, -1e-8, -0.01, -0.7, -3.0, -1e6]])
    c = Case("f32", [20, 13], [0, 4], 2, 2, 32, positions=[far + i for i in range(33)], inv_freq=f, seed=6)
    c.check(c.run())


@pytest.mark.parametrize("dtype", DTYPES)
def test_padding_rows_and_in_place_queries(dtype):
    """Rows behind the last sequence stay; queries may turn in place, inside the fused rows."""
    import torch
    c = Case(dtype, [4, 2], [1, 2], 4, 2, 64, pad=5, seed=5)
    before = c.fused.clone()
    k, v = c.k.clone(), c.v.clone()
    out = c.run(q_out=c.q)
    assert out.data_ptr() == c.q.data_ptr()
    c.check(out)
    assert torch.equal(c.fused[6:], before[6:])
    assert torch.equal(c.k, k) and torch.equal(c.v, v)
    c2 = Case(dtype, [4, 2], [1, 2], 4, 2, 64, pad=5, seed=5)
    fresh = c2.run()
    assert (fresh[6:] == 0).all() and torch.equal(fresh[:6], out[:6])


@pytest.mark.parametrize("dtype", DTYPES)
def test_without_queries_and_equal_shares(dtype):
    """No queries; and sequences of equal shares without offsets."""
    c = Case(dtype, [3, 3, 3], [1, 16, 0], 2, 2, 32, seed=6, with_q=False)
    assert c.run(seq_start=None) is None
    c.check()


def test_no_tokens_is_a_no_op():
    c = Case("bf16", [0, 0], [4, 5], 2, 2, 64, seed=7)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", DTYPES)
def test_replayed_graph(dtype):
    """A captured append replayed after lengths and offsets moved on."""
    import torch
    from transformer_encoder_gb300 import kv_append, sync_status
    a = Case(dtype, [1, 2, 1], [3, 4, 5], 2, 2, 64, page=8, seed=8)
    b = Case(dtype, [2, 0, 2], [7, 1, 0], 2, 2, 64, page=8, seed=9)
    pages, width = max(a.kc.shape[0], b.kc.shape[0]), max(a.table.shape[1], b.table.shape[1])
    fused = torch.empty_like(a.fused)
    kc = torch.zeros(pages, 8, 2, 64, dtype=a.kc.dtype, device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.zeros(3, width, dtype=torch.int32, device="cuda")
    lens, start = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    q_out = torch.empty_like(a.q)

    def fill(c):
        fused.copy_(c.fused)
        table.fill_(-1)
        table[:, :c.table.shape[1]].copy_(torch.from_numpy(c.table))
        lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        start.copy_(c.kw["seq_start"])
        kc.fill_(5.0)
        vc.fill_(6.0)

    step = lambda: kv_append(fused[:, 2:4], fused[:, 4:], kc, vc, table, lens, seq_start=start, q=fused[:, :2],
                             q_out=q_out, inv_freq=a.kw["inv_freq"])
    fill(a)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for c in (b, a):
        fill(c)
        g.replay()
        sync_status()
        c.kc, c.vc = kc, vc
        c.check(q_out)


@pytest.mark.parametrize("raw", [False, True])
def test_new_queries_on_another_stream(raw):
    """The tensor that is made for the queries is cleared in the order of the call's own stream, however
    busy the current one is."""
    import torch
    from transformer_encoder_gb300 import kv_append
    c = Case("bf16", [5, 9], [3, 0], 4, 2, 64, pad=3, seed=8)
    table, lens = torch.from_numpy(c.table).cuda(), torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)  # some 20 ms of the current stream
    out = kv_append(c.k, c.v, c.kc, c.vc, table, lens, stream=side.cuda_stream if raw else side, **c.kw)
    torch.cuda.synchronize()
    c.check(out)
    assert (out[c.n:] == 0).all()


def test_offsets_past_32_bits():
    """A page more than 2^32 bytes into the pool."""
    import torch
    from transformer_encoder_gb300 import kv_append, sync_status
    pages = (1 << 32) // (64 * 4 * 64 * 2) + 1
    kc = torch.zeros(pages, 64, 4, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    x = torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[0, pages - 1]], dtype=torch.int32, device="cuda")
    kv_append(x, x + 1, kc, vc, table, torch.tensor([127], dtype=torch.int32, device="cuda"))
    sync_status()
    assert torch.equal(kc[-1, 60:63], x) and torch.equal(vc[-1, 60:63], x + 1)
    assert int((kc[:-1] != 0).sum()) == 0


@pytest.mark.parametrize("what", ["page", "negative page", "table end", "short length", "offsets", "start"])
def test_bad_device_data_is_reported(what):
    """Page numbers, lengths and offsets out of range: reported, the tokens concerned left unwritten."""
    import torch
    from transformer_encoder_gb300 import WencError, kv_append, sync_status
    c = Case("bf16", [2, 3], [20, 3], 2, 2, 64, seed=10)
    table, lens = torch.from_numpy(c.table).cuda(), torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    start = c.kw["seq_start"].clone()
    if what == "page":
        table[0, 1] = c.kc.shape[0]
    if what == "negative page":
        table[0, 1] = -1
    if what == "table end":
        lens[0] = table.shape[1] * 16 + 1
    if what == "short length":
        lens[1] = 2  # three new tokens
    if what == "offsets":
        start[1] = 100
    if what == "start":
        start[0] = 1
    kv_append(c.k, c.v, c.kc, c.vc, table, lens, **{**c.kw, "seq_start": start})
    with pytest.raises(WencError, match="out of range") as e:
        sync_status()
    assert e.value.status == 1
    sync_status()  # cleared
