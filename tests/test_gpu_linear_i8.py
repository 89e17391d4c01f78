"""wenc_quantize_rows and wenc_linear_i8 against their definitions.

quantize_rows is exact: the integers are those of the exact quotient, bit for bit.
linear_i8: integer products are exact in fp32, and so are partial sums below 2^24; beyond that each of
the at most K additions rounds by 2^-23 (the tensor core may truncate) of a partial sum that is at
most S = sum |a||w| (in units of the scales). Scaling and bias: 4 roundings of 2^-24 of their operands.
  fp32 (residual): |err| <= 4 * 2^-24 (S' + |b| + |r|) + c S',  S' = S a_scale w_scale,
                   c = 0 for 127^2 K < 2^24, else K * 2^-23
  bf16: that, plus half a step of bf16 (2^-8); GELU: its slope is at most 1.13, and the erf formula
  adds 1.5e-7 |z| / 2 and the fp32 roundings of its evaluation (16 * 2^-24 |z|).
"""
import numpy as np
import pytest

import synth
from oracle import decode

pytestmark = pytest.mark.gpu


def _cuda(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ------------------------------------------------------------------ quantize_rows
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 16), (1, 384), (3, 48), (80, 1280), (7, 2032), (5, 5120), (2, 4112), (3, 20480), (2, 32784), (1, 65552),
                                    (1025, 512)])
def test_quantize_rows_is_exact(dtype, rows, d):
    import torch
    from transformer_encoder_gb300 import quantize_rows
    r = np.random.default_rng(rows * d)
    x = (r.standard_normal((rows, d)) * np.exp(2 * r.standard_normal((rows, 1)))).astype(np.float32)
    if dtype == "bf16":
        x = synth.round_to_bf16(x)
    t = _cuda(x)
    q, s = quantize_rows(t.to(torch.bfloat16) if dtype == "bf16" else t)
    want, scale = decode.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy(), scale)
    assert np.array_equal(q.cpu().numpy(), want)


def test_quantize_rows_at_its_edges():
    """Ties, zeros, one element, the smallest and largest numbers, infinities and NaN."""
    import torch
    from transformer_encoder_gb300 import quantize_rows
    d = 64
    x = np.zeros((16, d), np.float32)
    x[0, :] = np.arange(d) - 31.5          # scale 1 (amax 127): every value a tie
    x[0, 5] = 127.0
    x[1, 0] = -127.0
    x[1, 1:40] = np.arange(39) * 0.5
    x[3, 7] = 1e-45                        # the smallest subnormal
    x[4, :] = np.arange(d) * 1e-42
    x[5, :] = np.arange(d) * 2e-38
    x[6, :] = np.linspace(-3.4e38, 3.4e38, d)
    x[7, 3] = np.inf
    x[7, 4] = 1.0
    x[8, 3] = np.nan
    x[9, 63] = -np.inf
    x[10, :] = -5.0
    x[11, :] = np.nextafter(np.float32(0.5), np.float32(1)) * (1 + np.arange(d) % 3)
    x[11, 0] = 127.0
    x[12, :] = np.nextafter(np.float32(2.5), np.float32(0))
    x[12, 0] = 127.0
    x[13, :] = 1.2e-37 * np.arange(d)
    x[14, 0], x[14, 1] = 3.0, np.float32(1e-44)
    x[15, :] = (np.arange(d) + 0.5) * np.float32(2.0 ** -20)
    x[15, 0] = np.float32(127 * 2.0 ** -20)
    q, s = quantize_rows(_cuda(x))
    want, scale = decode.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy(), scale, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), want)
    xb = torch.full((2, 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    xb[1] = 0
    q, s = quantize_rows(xb)
    assert torch.isnan(s[0]) and s[1] == 0 and (q == 0).all()


def test_quantize_rows_past_32_bits():
    """More than 2^32 bytes of rows: the last ones are right."""
    import torch
    from transformer_encoder_gb300 import quantize_rows
    d = 8192
    rows = (1 << 32) // (2 * d) + 3
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, d, device="cuda").to(torch.bfloat16)
    q, s = quantize_rows(x)
    want, scale = decode.quantize_rows(x[-3:].float().cpu().numpy())
    assert np.array_equal(q[-3:].cpu().numpy(), want) and np.array_equal(s[-3:].cpu().numpy(), scale)
    assert int((s[:-3] != 0).sum()) == 0


# ------------------------------------------------------------------ linear_i8
def _gelu(z):
    from math import erf
    return z * 0.5 * (1 + np.vectorize(erf)(z * np.sqrt(0.5)))


def _problem(M, N, K, seed=0, extreme=False):
    r = np.random.default_rng(seed)
    if extreme:
        a = np.full((M, K), 127, np.int8)
        w = np.where(r.random((N, 1)) < 0.5, 127, -127).astype(np.int8) * np.ones((1, K), np.int8)
    else:
        a = np.clip(np.rint(r.standard_normal((M, K)) * 40), -127, 127).astype(np.int8)
        w = np.clip(np.rint(r.standard_normal((N, K)) * 40), -127, 127).astype(np.int8)
    sa = np.exp(r.standard_normal(M)).astype(np.float32) * 0.02
    sw = (np.exp(0.3 * r.standard_normal(N)) * 0.5 / (40 * np.sqrt(K))).astype(np.float32)
    b = (0.1 * r.standard_normal(N)).astype(np.float32)
    return a, sa, w, sw, b, r.standard_normal((M, N)).astype(np.float32)


def _check(got, a, sa, w, sw, b, resid, epilogue, what):
    K = a.shape[1]
    z, mag = decode.linear_i8(a, sa, w, sw, b)
    c = 0.0 if 127 * 127 * K < 1 << 24 else K * 2.0 ** -23
    slack = 4 * 2.0 ** -24 * (mag + np.abs(b)) + c * mag
    if epilogue == 2:
        ref = z + resid
        bound = slack + 4 * 2.0 ** -24 * np.abs(resid)
    elif epilogue == 1:
        ref = _gelu(z)
        slack = 1.13 * slack + (0.75e-7 + 16 * 2.0 ** -24) * np.abs(z)
        bound = slack + 2.0 ** -8 * (np.abs(ref) + slack)
    else:
        ref = z
        bound = slack + 2.0 ** -8 * (np.abs(ref) + slack)
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    assert (err <= bound + 1e-30).all(), f"{what}: {float((err / (bound + 1e-30)).max()):.2f} x the bound"


def _run(a, sa, w, sw, b, resid, epilogue, **kw):
    from transformer_encoder_gb300 import linear_i8, sync_status
    out = linear_i8(_cuda(a), _cuda(sa), _cuda(w), _cuda(sw), _cuda(b), epilogue,
                    resid=_cuda(resid) if epilogue == 2 else None, **kw)
    sync_status()
    return out


@pytest.mark.parametrize("epilogue", [0, 1, 2])
@pytest.mark.parametrize("M,N,K", [(1, 128, 64), (1, 1536, 384), (5, 384, 128), (16, 256, 1280), (17, 640, 192),
                                   (33, 1280, 320), (80, 1152, 1280), (127, 512, 576), (129, 128, 2048),
                                   (300, 384, 1536), (1537, 1152, 384), (513, 2560, 640),
                                   (18, 128, 64), (31, 128, 8192), (128, 256, 320), (100, 5120, 1280), (2049, 256, 448)])
def test_linear_i8(M, N, K, epilogue):
    p = _problem(M, N, K, seed=M + N + K)
    _check(_run(*p, epilogue).double().cpu().numpy(), *p, epilogue, f"{M} x {N} x {K}")


@pytest.mark.parametrize("epilogue", [0, 2])
@pytest.mark.parametrize("M,N,K", [(3, 20608, 64), (17, 20608, 64), (128, 19584, 192), (129, 10240, 1088), (250, 9984, 1024),
                                   (250, 10240, 192), (300, 19584, 128)])
def test_linear_i8_many_channels(M, N, K, epilogue):
    """More output tiles than SMs, from few tokens: in every form."""
    p = _problem(M, N, K, seed=M)
    _check(_run(*p, epilogue).double().cpu().numpy(), *p, epilogue, f"{M}x{N}x{K}")


@pytest.mark.parametrize("M", [1, 8, 40, 200])
def test_linear_i8_largest_sums(M):
    """All products 127^2 of one sign: sums far beyond 2^24."""
    p = _problem(M, 256, 5120, seed=M, extreme=True)
    _check(_run(*p, 2).double().cpu().numpy(), *p, 2, f"extreme M = {M}")


def test_linear_i8_takes_the_lowest_integer():
    """-128 is no output of quantize_rows, but an int8 weight may hold it."""
    for M in (3, 300):
        a, sa, w, sw, b, r = _problem(M, 128, 128, seed=9)
        a[:, ::3] = -128
        w[::2] = -128
        _check(_run(a, sa, w, sw, b, r, 2).double().cpu().numpy(), a, sa, w, sw, b, r, 2, f"-128, M = {M}")


@pytest.mark.parametrize("M", [2, 40, 300])
def test_linear_i8_nan_scale_stays_in_its_row(M):
    """A row whose activations were not finite has scale NaN: its outputs are NaN, no others."""
    a, sa, w, sw, b, r = _problem(M, 256, 128, seed=3)
    sa[1] = np.nan
    a[1] = 0
    got = _run(a, sa, w, sw, b, r, 2).double().cpu().numpy()
    assert np.isnan(got[1]).all()
    keep = np.arange(M) != 1
    _check(got[keep], a[keep], sa[keep], w, sw, b, r[keep], 2, "others")


@pytest.mark.parametrize("M", [3, 70, 400])
def test_linear_i8_in_place_residual_graph_and_stream(M):
    """out may be resid; a captured call replays; another stream."""
    import torch
    from transformer_encoder_gb300 import linear_i8, sync_status
    p = _problem(M, 384, 256, seed=4)
    a, sa, w, sw, b = (_cuda(x) for x in p[:5])
    want = _run(*p, 2)
    x = _cuda(p[5])
    linear_i8(a, sa, w, sw, b, 2, resid=x, out=x)
    sync_status()
    assert torch.equal(x, want)
    r0 = _cuda(p[5])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = linear_i8(a, sa, w, sw, b, 2, resid=r0, stream=s)
    sync_status()
    assert torch.equal(out, want)
    r = _cuda(p[5])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = linear_i8(a, sa, w, sw, b, 2, resid=r)
    for k in (1.0, 0.0):
        r.copy_(_cuda(p[5]) * k)
        g.replay()
        sync_status()
        _check(out.double().cpu().numpy(), *p[:5], p[5] * np.float32(k), 2, "replayed")


def test_every_token_count_around_the_tiles():
    """Token counts 1 .. 33 and around 128 and 256: no column of the MMA's padding reaches the output."""
    import torch
    a, sa, w, sw, b, r = _problem(260, 128, 192, seed=12)
    for M in list(range(1, 34)) + [63, 64, 65, 112, 113, 127, 128, 129, 255, 256, 257, 260]:
        got = _run(a[:M], sa[:M], w, sw, b, r[:M], 2).double().cpu().numpy()
        _check(got, a[:M], sa[:M], w, sw, b, r[:M], 2, f"M = {M}")


def test_outputs_past_32_bits():
    """More than 2^32 bytes of output and of tokens' rows: the last ones are right."""
    import torch
    M, N, K = (1 << 32) // (2 * 1024) + 130, 1024, 128
    a = torch.zeros(M, K, dtype=torch.int8, device="cuda")
    p = _problem(130, N, K, seed=13)
    a[-130:] = _cuda(p[0])
    sa = torch.ones(M, device="cuda")
    sa[-130:] = _cuda(p[1])
    from transformer_encoder_gb300 import linear_i8, sync_status
    out = linear_i8(a, sa, _cuda(p[2]), _cuda(p[3]), _cuda(p[4]), 0)
    sync_status()
    _check(out[-130:].double().cpu().numpy(), *p, 0, "last rows")
    assert torch.equal(out[0], _cuda(p[4]).to(torch.bfloat16)) and torch.equal(out[M - 131], out[0])


@pytest.mark.parametrize("epilogue", [0, 2])
def test_a_given_workspace(epilogue):
    """The two-pass form in a given workspace of any content; one that is too small is refused."""
    import torch
    from transformer_encoder_gb300 import WencError, lib, linear_i8, sync_status
    M, N, K = 7777, 512, 1024
    p = _problem(M, N, K, seed=14)
    d = [_cuda(x) for x in p]
    need = lib().wenc_linear_i8_workspace(M, N, K)
    assert need >= 2 * K * (M + N)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = linear_i8(*d[:5], epilogue, resid=d[5] if epilogue == 2 else None, workspace=ws)
    sync_status()
    rows = np.unique(np.r_[0, 255, 256, M - 1, np.random.default_rng(0).integers(0, M, 60)])
    _check(out[torch.from_numpy(rows).cuda()].double().cpu().numpy(), p[0][rows], p[1][rows], p[2], p[3], p[4], p[5][rows],
           epilogue, "given workspace")
    with pytest.raises(WencError, match="workspace"):
        linear_i8(*d[:5], 0, workspace=ws[:need - 256])


@pytest.mark.parametrize("M", [5, 2000])
def test_two_streams_at_once(M):
    import torch
    from transformer_encoder_gb300 import linear_i8
    ps = [_problem(M, 512, 640, seed=s) for s in (5, 6)]
    dev = [[_cuda(x) for x in p[:5]] for p in ps]
    want = [_run(*p, 0) for p in ps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for d, s, k in zip(dev, streams, (0, 1)):
            with torch.cuda.stream(s):
                outs.append((k, linear_i8(*d, 0)))
    torch.cuda.synchronize()
    for k, o in outs:
        assert torch.equal(o, want[k])


def test_quantized_layer_is_near_the_full_one():
    """quantize_rows and linear_i8 as they are used, against the unquantised product: each operand is
    off by at most half its scale."""
    import torch
    from transformer_encoder_gb300 import linear_i8, quantize_rows, sync_status
    r = np.random.default_rng(0)
    M, N, K = 77, 256, 512
    x, w = r.standard_normal((M, K)).astype(np.float32), (0.05 * r.standard_normal((N, K))).astype(np.float32)
    wq, sw = quantize_rows(_cuda(w))
    xq, sx = quantize_rows(_cuda(x))
    out = linear_i8(xq, sx, wq, sw, torch.zeros(N, device="cuda"), 2, resid=torch.zeros(M, N, device="cuda"))
    sync_status()
    sx, sw = sx.cpu().numpy().astype(np.float64), sw.cpu().numpy().astype(np.float64)
    dx, dw = 0.5 * sx[:, None], 0.5 * sw[:, None]
    bound = dx * np.abs(w).sum(1)[None] + np.abs(x).sum(1)[:, None] * dw.T + K * dx * dw.T
    ref = x.astype(np.float64) @ w.astype(np.float64).T
    assert (np.abs(out.double().cpu().numpy() - ref) <= 1.0001 * bound).all()
