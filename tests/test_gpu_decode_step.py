"""The decode-side operators together, as a program uses them after the encoder: one decoder layer's
attention half over beams, eager and captured, for several tokens.

x (the residual stream) -> 8-bit Q/K/V projection -> append to the paged cache with rotation ->
attention over the shared prompt and the own pages -> 8-bit out-projection onto the stream; then the
cross-attention of the result's queries over the planes that Encoder.cross_kv wrote. Every stage's
output is compared with the float64 definition on the GPU's own inputs of that stage, so the bounds are
those of the single operators (see their tests): here as relative L2, half a step of bf16 (2^-8) for
the bf16 stages and 2^-18 for the fp32 output.
"""
import numpy as np
import pytest

import synth
from helpers import make_encoder
from oracle import decode

pytestmark = pytest.mark.gpu

B, BEAMS, H, D, PAGE, STEPS = 2, 3, 6, 384, 4, 6
N = B * BEAMS


def _near(got, ref, tol, what):
    got = got.double().cpu().numpy().reshape(ref.shape)
    assert np.isfinite(got).all(), what
    assert np.linalg.norm(got - ref) <= tol * np.linalg.norm(ref), (what, np.linalg.norm(got - ref) / np.linalg.norm(ref))


def test_decode_steps_over_encoder_planes():
    import torch
    import transformer_encoder_gb300 as wenc
    w = synth.WORKLOADS["tiny_stack"]
    enc, _, _, rng = make_encoder(w, keep_host_layers=False, max_batch=B)
    dec = synth.make_cross(w, 2)
    up = lambda a, t=None: torch.from_numpy(np.ascontiguousarray(a)).cuda().to(t or torch.float32)
    enc.set_cross_kv([{"wk": up(p["wk"], torch.bfloat16), "wv": up(p["wv"], torch.bfloat16), "bv": up(p["bv"])} for p in dec])
    r = np.random.default_rng(3)
    y = enc.forward(up(r.standard_normal((B, w.seq_len, D)).astype(np.float32)))
    planes = enc.cross_kv(y).view(2, 2, B, w.seq_len, H, 64)  # [layer, K or V, window, frame, head, 64]

    wqkv, s_qkv = wenc.quantize_rows(up(0.05 * r.standard_normal((3 * D, D))))
    wo, s_o = wenc.quantize_rows(up(0.05 * r.standard_normal((D, D))))
    b_qkv, b_o = up(0.01 * r.standard_normal(3 * D)), up(0.01 * r.standard_normal(D))
    freq = up([10000.0 ** (-2.0 * i / 64) for i in range(32)])
    prompt = up(r.standard_normal((2, B, 9, H, 64)), torch.bfloat16)
    prompt_lens = torch.tensor([9, 4], dtype=torch.int32, device="cuda")
    pages = torch.full((2, N * 3, PAGE, H, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    table = torch.from_numpy(r.permutation(N * 3).reshape(N, 3).astype(np.int32)).cuda()
    lens = torch.zeros(N, dtype=torch.int32, device="cuda")
    position = torch.zeros(N, dtype=torch.int32, device="cuda")
    x = torch.zeros(N, D, device="cuda")

    def step():
        xq, sx = wenc.quantize_rows(x)
        qkv = wenc.linear_i8(xq, sx, wqkv, s_qkv, b_qkv, wenc.EPI_BIAS_BF16).view(N, 3 * H, 64)
        lens.add_(1)
        turned = wenc.kv_append(qkv[:, H:2 * H], qkv[:, 2 * H:], pages[0], pages[1], table, lens, q=qkv[:, :H],
                                positions=position, inv_freq=freq)
        o = wenc.prefix_attention(turned.view(N, 1, H, 64), prompt[0], prompt[1], prefix_lens=prompt_lens, k_pages=pages[0],
                                  v_pages=pages[1], block_table=table, lens=lens)
        oq, so = wenc.quantize_rows(o.view(N, D))
        z = wenc.linear_i8(oq, so, wo, s_o, b_o, wenc.EPI_BIAS_RESID_F32, resid=x)
        cross = wenc.prefix_attention(z.to(torch.bfloat16).view(N, 1, H, 64), planes[1, 0], planes[1, 1])
        return xq, sx, qkv, turned, o, oq, so, z, cross

    host = lambda t: t.double().cpu().numpy()
    groups = [g for g in range(B) for _ in range(BEAMS)]
    cross_kv = [(host(planes[1, 0, b]), host(planes[1, 1, b])) for b in range(B)]
    prompts = [(host(prompt[0, b, :m]), host(prompt[1, b, :m])) for b, m in enumerate((9, 4))]

    def check(t, out):
        xq, sx, qkv, turned, o, oq, so, z, cross = out
        ints, scale = decode.quantize_rows(x.cpu().numpy())
        assert np.array_equal(xq.cpu().numpy(), ints) and np.array_equal(sx.cpu().numpy(), scale)
        ref, _ = decode.linear_i8(ints, scale, wqkv.cpu().numpy(), s_qkv.cpu().numpy(), b_qkv.cpu().numpy())
        _near(qkv, ref, 2.0 ** -8, "qkv")
        q3, pos = host(qkv), position.cpu().numpy()
        _near(turned, decode.rotate(q3[:, :H], pos, freq.cpu().numpy(), False)[0], 2.0 ** -8, "queries")
        k, v, tab = host(pages[0]), host(pages[1]), table.cpu().numpy()
        owns = []
        for s in range(N):
            at = np.arange(t + 1)
            owns.append((k[tab[s, at // PAGE], at % PAGE], v[tab[s, at // PAGE], at % PAGE]))
            assert np.array_equal(owns[-1][1][-1], q3[s, 2 * H:])
        newest = np.stack([own[0][-1] for own in owns])
        _near(torch.from_numpy(newest), decode.rotate(q3[:, H:2 * H], pos, freq.cpu().numpy(), False)[0], 2.0 ** -8, "keys")
        ref, _, _ = decode.prefix_attention(host(turned)[:, None], prompts, owns, groups)
        _near(o, ref, 2.0 ** -8, "self-attention")
        ints, scale = decode.quantize_rows(o.float().cpu().numpy().reshape(N, D))
        assert np.array_equal(oq.cpu().numpy(), ints) and np.array_equal(so.cpu().numpy(), scale)
        ref, _ = decode.linear_i8(ints, scale, wo.cpu().numpy(), s_o.cpu().numpy(), b_o.cpu().numpy())
        _near(z, ref + host(x), 2.0 ** -18, "out-projection")
        zq = host(z.to(torch.bfloat16)).reshape(N, 1, H, 64)
        empty = [(np.zeros((0, H, 64)),) * 2] * N
        _near(cross, decode.prefix_attention(zq, cross_kv, empty, groups)[0], 2.0 ** -8, "cross-attention")

    def enter(t):
        x.copy_(up(np.random.default_rng(100 + t).standard_normal((N, D))))
        position.copy_(prompt_lens.repeat_interleave(BEAMS) + t)

    for t in range(2):  # eager
        enter(t)
        out = step()
        wenc.sync_status()
        check(t, out)
    g = torch.cuda.CUDAGraph()
    saved = lens.clone()
    with torch.cuda.graph(g):
        out = step()
    lens.copy_(saved)
    for t in range(2, STEPS):  # replayed
        enter(t)
        g.replay()
        wenc.sync_status()
        check(t, out)
    assert lens.tolist() == [STEPS] * N
