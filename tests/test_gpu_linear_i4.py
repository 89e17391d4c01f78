"""wenc_linear_i4 against its definition in 64 bits, over types, group sizes, epilogues and numbers of tokens.

Let S = sum_g |scale_g| sum_{k in g} |u - 8| |x_k|. bf16 products with integers are exact in fp32; a group's at most 128 of
them accumulate with a rounding of 2^-23 each (the tensor core may truncate), float32 x three parts of them: 3 * 128. The
groups' sums and their join over warps and CTAs: K / 32 + 64 roundings of 2^-24 at most. Bias and residual: 2^-24 each.
  |err| <= (c * 2^-23 + (K / 32 + 64) 2^-24) S + 3 * 2^-24 (S + |b| + |r|),   c = 128 (bf16 x), 384 (float32 x)
bf16 output: plus half a step, 2^-8 of the value; GELU: its slope is at most 1.13, and erf's approximation and the fp32 roundings of
its evaluation add at most 1.5e-7 |z| / 2 + 16 * 2^-24 |z|.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, M, N, K, group, x="bf16", scale="bf16", epilogue=0, seed=0):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        dt = {"bf16": torch.bfloat16, "f32": torch.float32}
        self.x = (torch.randn(M, K, generator=g, device="cuda") * torch.exp(torch.randn(M, 1, generator=g, device="cuda"))).to(dt[x])
        self.w = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        self.scale = (torch.exp(0.5 * torch.randn(N, K // group, generator=g, device="cuda")) * 0.01).to(dt[scale])
        self.scale[::3] *= -1
        self.bias = torch.randn(N, generator=g, device="cuda")
        self.resid = torch.randn(M, N, generator=g, device="cuda")
        self.epilogue, self.group = epilogue, group

    def run(self, **kw):
        from transformer_encoder_gb300 import linear_i4, sync_status
        out = linear_i4(self.x, self.w, self.scale, self.bias, self.epilogue, resid=self.resid if self.epilogue == 2 else None, **kw)
        sync_status()
        return out

    def check(self, out):
        import torch
        u = torch.stack([self.w & 15, self.w >> 4], 2).flatten(1).double() - 8.0
        w = u * self.scale.double().repeat_interleave(self.group, 1)
        x, K = self.x.double(), self.x.shape[1]
        z, S = x @ w.t() + self.bias.double(), x.abs() @ w.abs().t()
        f32 = self.x.dtype is torch.float32
        r = self.resid.double() if self.epilogue == 2 else torch.zeros_like(z)
        bound = ((384 if f32 else 128) * 2.0 ** -23 + (K / 32 + 64) * 2.0 ** -24) * S + 3 * 2.0 ** -24 * (S + self.bias.double().abs() + r.abs())
        ref = z + r
        if self.epilogue == 1:
            ref = z * torch.special.ndtr(z)
            bound = 1.13 * bound + (0.75e-7 + 16 * 2.0 ** -24) * z.abs()
        if out.dtype is torch.bfloat16:
            bound = bound * 1.01 + 2.0 ** -8 * ref.abs()
        assert out.dtype is (torch.float32 if self.epilogue == 2 or f32 else torch.bfloat16)
        err = (out.double() - ref).abs()
        assert torch.isfinite(out).all() and (err <= bound + 1e-30).all(), float((err / (bound + 1e-30)).max())
        limit = 2.0 ** -8 if out.dtype is torch.bfloat16 else 2.0 ** -19
        assert float((out.double() - ref).norm()) <= limit * float(ref.norm())


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 17, 33, 80, 127, 129, 300])
def test_tokens_and_groups(x, group, M):
    c = Case(M, 384, 640, group, x, "f32" if M % 2 else "bf16", seed=M)
    c.check(c.run())


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("scale", ["bf16", "f32"])
@pytest.mark.parametrize("epilogue", [0, 1, 2])
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (5, 1152, 384), (80, 5120, 1280), (700, 256, 1280), (40, 128, 5120), (2, 128, 8064)])
def test_epilogues_and_types(x, scale, epilogue, M, N, K):
    c = Case(M, N, K, 64, x, scale, epilogue, seed=N + K)
    c.check(c.run())


@pytest.mark.parametrize("M", [1, 200])
def test_residual_in_place(M):
    import torch
    from transformer_encoder_gb300 import linear_i4
    c = Case(M, 256, 512, 128, epilogue=2)
    want = c.run()
    stream = c.resid.clone()
    assert linear_i4(c.x, c.w, c.scale, c.bias, 2, resid=stream, out=stream) is stream
    assert torch.equal(stream, want)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("M", [4, 150])
def test_inputs_that_are_no_numbers_stay_in_their_rows(x, M):
    """An infinity or a NaN in a token reaches that token's outputs alone; the largest numbers stay numbers."""
    import torch
    c = Case(M, 256, 256, 32, x)
    want = c.run()
    c.w &= 0x77  # (weights of -8 .. -1: no 0 x inf)
    clean = c.run()
    c.x[1, 77], c.x[2, 5], c.x[3, 9] = float("nan"), float("inf"), -float("inf")
    got = c.run()
    rest = [m for m in range(M) if m not in (1, 2, 3)]
    assert torch.equal(got[rest], clean[rest]) and torch.isnan(got[1]).all()
    neg = c.scale[:, 0] < 0
    assert (got[2][neg] == float("inf")).all() and (got[2][~neg] == -float("inf")).all()
    assert (got[3][neg] == -float("inf")).all() and (got[3][~neg] == float("inf")).all()
    assert want.shape == got.shape
    if x == "f32":
        c.x.fill_(0.0)
        c.x[:, 40] = 3.4028234e38
        c.scale.fill_(2.0 ** -9)
        c.w.fill_(0x99)
        out = c.run()
        assert (out.double() - (c.x[:, 40:41].double() * 2.0 ** -9 + c.bias.double())).abs().max() <= 2.0 ** -23 * 3.4e38 * 2.0 ** -9


def test_every_weight_and_its_place():
    """Unit inputs read single weights: all sixteen values at every position of a piece."""
    import torch
    from transformer_encoder_gb300 import linear_i4
    N, K = 128, 256
    u = (torch.arange(N, device="cuda").view(N, 1) * 7 + torch.arange(K, device="cuda").view(1, K) * 3) % 16
    w = (u[:, 0::2] | (u[:, 1::2] << 4)).to(torch.uint8)
    scale = torch.ones(N, K // 32, device="cuda") * torch.tensor([1.0, 2.0, 4.0, 8.0] * 2, device="cuda")
    for M in (8, 256):
        x = torch.eye(K, device="cuda", dtype=torch.bfloat16)
        want = (u.float() - 8).t() * scale.repeat_interleave(32, 1).t()
        got = torch.cat([linear_i4(x[i:i + M].contiguous(), w, scale, torch.zeros(N, device="cuda")) for i in range(0, K, M)])
        assert torch.equal(got.float(), want)


def test_streams_and_graphs():
    import torch
    from transformer_encoder_gb300 import linear_i4, sync_status
    for M in (3, 180):
        for x in ("bf16", "f32"):
            c = Case(M, 384, 1280, 64, x, epilogue=1)
            want = c.run()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            out = linear_i4(c.x, c.w, c.scale, c.bias, 1, stream=side)
            side.synchronize()
            assert torch.equal(out, want)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = linear_i4(c.x, c.w, c.scale, c.bias, 1)
            c.x.mul_(0.5)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, c.run())
    sync_status()


def test_what_the_binding_refuses():
    import torch
    from transformer_encoder_gb300 import linear_i4
    c = Case(4, 256, 256, 64)
    a = [c.x, c.w, c.scale, c.bias]
    for i, bad in ((0, c.x.half()), (0, c.x[:, :128]), (0, c.x[0]), (0, c.x.cpu()), (0, c.x.t().contiguous().t()), (1, c.w.to(torch.int8)),
                   (1, c.w[:, :64]), (2, c.scale.half()), (2, c.scale[:, :3]), (2, c.scale[:, :1]), (2, c.scale[:8]), (3, c.bias.half()),
                   (3, c.bias[:8])):
        with pytest.raises(Exception):
            linear_i4(*[bad if j == i else y for j, y in enumerate(a)])
    for kw in (dict(epilogue=3), dict(epilogue=2), dict(epilogue=2, resid=c.resid.half()), dict(out=torch.empty(4, 256, device="cuda"))):
        with pytest.raises(Exception):
            linear_i4(*a, **kw)
    assert linear_i4(c.x[:0], *a[1:]).shape == (0, 256)


@pytest.mark.parametrize("x,M,N", [("bf16", (1 << 21) + 77, 1152), ("f32", (1 << 20) + 5, 2304)])
def test_offsets_past_32_bits(x, M, N):
    """More than 2^31 results. Whole numbers of which every sum is exact, so any division of the rows gives the same bits."""
    import torch
    from transformer_encoder_gb300 import linear_i4, sync_status
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    assert M * N > 1 << 31
    a = torch.randint(-3, 4, (M, 128), generator=g, device="cuda").to(torch.bfloat16 if x == "bf16" else torch.float32)
    w = torch.randint(0, 256, (N, 64), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.full((N, 2), 0.125, device="cuda")
    b = torch.zeros(N, device="cuda")
    out = linear_i4(a, w, s, b)
    for lo in (0, M // 2 - 40, M - 300):
        assert torch.equal(out[lo:lo + 300], linear_i4(a[lo:lo + 300], w, s, b))
    u = torch.stack([w & 15, w >> 4], 2).view(N, 128).double() - 8
    want = (a[-8:].double() @ u.t() * 0.125).to(out.dtype)
    assert torch.equal(out[-8:], want)
    sync_status()
