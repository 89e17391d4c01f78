"""The decode-side operators, as they are measured: what a program that has run the encoder calls next.

- prefix_attention: the queries of sequences that share a prefix (the beams of a window over its cross keys, prompts of a
  batch) against the shared keys and each sequence's own keys in a paged cache.
- kv_append: new keys and values into that cache, with the position rotation of keys and queries.
- linear_i8: quantize_rows and the product in 8-bit integers with a scale for each token and each channel.

The plain forms are elementary torch operations in 32 bits (angles and quantisation borders in 64).
"""
import math
import random

import numpy as np
import torch

own = False

HD = 64  # the framework's head width
GELU, RESID = 1, 2  # epilogues; 0 is the bias alone

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _attn(name, dtype, groups, beams, q_len, heads, kv_heads, prefix, suffix, page, ragged, uneven, strided, shape):
    return dict(name=name, op="prefix_attention", dtype=dtype, groups=groups, beams=beams, q_len=q_len, heads=heads,
                kv_heads=kv_heads, prefix=prefix, suffix=suffix, page=page, ragged=ragged, uneven=uneven,
                strided=strided, shape=shape)


def _append(name, dtype, seqs, max_new, heads, kv_heads, rot, interleaved, past, page, ragged, pad, far, shape):
    return dict(name=name, op="kv_append", dtype=dtype, seqs=seqs, max_new=max_new, heads=heads, kv_heads=kv_heads,
                rot=rot, interleaved=interleaved, past=past, page=page, ragged=ragged, pad=pad, far=far, shape=shape)


def _i8(name, x, M, N, K, epilogue):
    return dict(name=name, op="linear_i8", x=x, M=M, N=N, K=K, epilogue=epilogue)


def listed():
    return [
        # greedy decoding of one window at the tiny dims: one query token over the window's cross keys
        _attn("cross_greedy_tiny", "bf16", 1, 1, 1, 6, 6, 1500, 0, 16, False, False, False, 1),
        # beam search at the large dims: 16 windows x 5 beams over the cross keys of one decoder layer
        _attn("cross_beams_large", "bf16", 16, 5, 1, 20, 20, 1500, 0, 16, False, False, False, 2),
        # the same beams' self-attention: prompts of up to 224 tokens shared by a window's beams (some have none),
        # own tokens in pages of 16; windows have lost some of their beams; q is a slice of the fused projection
        _attn("self_beams_large", "bf16", 16, 5, 1, 20, 20, 224, 224, 16, True, True, True, 3),
        # 256 sequences behind one long prompt, 4 key heads for 20 query heads, up to 600 own tokens in pages of 64
        _attn("long_prompt_shared", "bf16", 1, 256, 1, 20, 4, 8191, 600, 64, True, False, False, 4),
        # fp32 planes (the TF32 precision), base dims: 4 windows x 5 beams, 3 draft tokens a step, odd pages
        _attn("drafts_base_f32", "f32", 4, 5, 3, 8, 8, 1500, 100, 24, True, False, True, 5),
        # one token of one sequence, tiny dims (latency)
        _append("append_one_tiny", "bf16", 1, 1, 6, 6, 64, False, 100, 16, False, 0, 0, 6),
        # the prompts of 16 sequences at once, ragged, 4 key heads for 20 query heads, with padding rows behind them
        _append("append_prompts", "bf16", 16, 4000, 20, 4, 64, False, 0, 64, True, 77, 0, 7),
        # chunks of up to 33 tokens of 80 sequences far into long streams, fp32, half of each head rotated in
        # neighbouring pairs, odd pages
        _append("append_far_f32", "f32", 80, 33, 8, 8, 32, True, 400, 24, True, 5, 1000000, 8),
        # one token through fc1 of the tiny dims
        _i8("fc1_one_tiny", "f32", 1, 1536, 384, GELU),
        # one step of 16 windows x 5 beams through fc1 of the large dims
        _i8("fc1_beams_large", "bf16", 80, 5120, 1280, GELU),
        # one window through the base dims' fused projection, ragged rows
        _i8("qkv_window_base", "f32", 1500, 1536, 512, 0),
        # 16 windows through fc2 of the large dims, onto the residual stream
        _i8("fc2_windows_large", "bf16", 24000, 1280, 5120, RESID),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _seconds(case):
    w = work(case)
    return w["bytes"] / 6.8e12 + w["flops"] / 1.9e15


def draw(rng):
    op = rng.choice(["prefix_attention", "prefix_attention", "kv_append", "linear_i8"])
    most = max(_seconds(c) for c in listed() if c["op"] == op)
    while True:
        shape = rng.randrange(1 << 30)
        if op == "prefix_attention":
            dtype = rng.choice(["bf16", "bf16", "f32"])
            heads, kv = rng.choice([(6, 6), (8, 8), (12, 12), (20, 20), (20, 4), (16, 2), (5, 1), (8, 4)])
            if rng.random() < 0.6:  # windows with beams
                groups, beams = _log(rng, 1, 16), rng.randint(1, 8)
                prefix = rng.choice([1500, _log(rng, 1, 1500), _log(rng, 1, 1500)])
            else:  # many behind one prompt
                groups, beams = rng.randint(1, 2), _log(rng, 9, 256)
                prefix = _log(rng, 16, 8191)
            q_len = rng.choice([1, 1, 1, 2, 3, 5, 8])
            suffix = rng.choice([0, _log(rng, 8, 600), _log(rng, 8, 600)])
            c = _attn(None, dtype, groups, beams, q_len, heads, kv, prefix, suffix, rng.choice([8, 16, 24, 64]),
                      rng.random() < 0.6, beams > 1 and rng.random() < 0.4, rng.random() < 0.5, shape)
        elif op == "kv_append":
            heads, kv = rng.choice([(6, 6), (8, 8), (12, 12), (20, 20), (20, 4), (16, 2), (5, 1)])
            c = _append(None, rng.choice(["bf16", "bf16", "f32"]), _log(rng, 1, 128), _log(rng, 1, 4000), heads, kv,
                        rng.choice([0, 16, 32, 64, 64]), rng.random() < 0.4, _log(rng, 1, 2000) - 1,
                        rng.choice([8, 16, 24, 64]), rng.random() < 0.6, rng.choice([0, 1, 30]),
                        rng.choice([0, _log(rng, 1000, 1000000)]), shape)
        else:
            c = _i8(None, rng.choice(["bf16", "f32"]), _log(rng, 1, 24000), 128 * _log(rng, 3, 40),
                    64 * _log(rng, 6, 80), rng.choice([0, GELU, RESID]))
        del c["name"]
        if _seconds(c) <= most:
            return c


# ------------------------------------------------------------------ what the cases' lengths are
def _attn_lens(case):
    """(group sizes, prefix lengths, own lengths with the step's tokens)"""
    r = random.Random(case["shape"])
    G, S, t = case["groups"], case["beams"], case["q_len"]
    sizes = [r.randint(1, S) if case["uneven"] else S for _ in range(G)]
    sizes[r.randrange(G)] = S
    n = sum(sizes)
    if case["ragged"]:
        pre = [r.randint(0, case["prefix"]) for _ in range(G)]
        pre[r.randrange(G)] = case["prefix"]
        suf = [r.randint(min(t, case["suffix"]), case["suffix"]) for _ in range(n)]
    else:
        pre, suf = [case["prefix"]] * G, [case["suffix"]] * n
    return sizes, pre, suf


def _append_lens(case):
    """(new tokens, lengths with them) of each sequence"""
    r = random.Random(case["shape"])
    n = case["seqs"]
    new = [r.randint(0, case["max_new"]) if case["ragged"] else case["max_new"] for _ in range(n)]
    new[r.randrange(n)] = case["max_new"]
    return new, [(r.randint(0, case["past"]) if case["ragged"] else case["past"]) + m for m in new]


def _seen(length, t):
    """own keys that t tokens at the end of `length` see, together"""
    return sum(max(0, length - t + 1 + i) for i in range(t))


def work(case):
    if case["op"] == "prefix_attention":
        sizes, pre, suf = _attn_lens(case)
        e = 2 if case["dtype"] == "bf16" else 4
        n, t, H, kv = sum(sizes), case["q_len"], case["heads"], case["kv_heads"]
        keys = sum(p * s * t for p, s in zip(pre, sizes)) + sum(_seen(v, t) for v in suf)
        return {"bytes": e * HD * (2 * n * t * H + 2 * kv * (sum(pre) + sum(suf))), "flops": 4 * HD * H * keys}
    if case["op"] == "kv_append":
        new, _ = _append_lens(case)
        e = 2 if case["dtype"] == "bf16" else 4
        n, H, kv = sum(new), case["heads"], case["kv_heads"]
        return {"bytes": 2 * e * HD * n * (H + 2 * kv), "flops": 3 * case["rot"] * n * (H + kv)}
    M, N, K = case["M"], case["N"], case["K"]
    e = 2 if case["x"] == "bf16" else 4
    return {"bytes": e * M * K + N * K + (8 if case["epilogue"] == RESID else 2) * M * N + 8 * N,
            "flops": 2 * M * N * K}


# ------------------------------------------------------------------ what the program has in hand
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pages(g, lens, page, kv, dtype):
    """A pool with the pages of all sequences in shuffled order and a table of them (-1 behind a sequence's last)."""
    need = np.array([-(-v // page) for v in lens])
    width, total = max(1, int(need.max())), max(1, int(need.sum()))
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.from_numpy((np.cumsum(need) - need)[:, None] + np.arange(width)).cuda()
    there = torch.from_numpy(np.arange(width) < need[:, None]).cuda()
    table = torch.where(there, order[at.clamp(max=total - 1)], -1)
    pool = [torch.randn(total, page, kv, HD, generator=g, device="cuda").to(dtype) for _ in range(2)]
    return pool[0], pool[1], table


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = {"case": case}
    if case["op"] == "prefix_attention":
        sizes, pre, suf = _attn_lens(case)
        dt, n, t, H, kv = DT[case["dtype"]], sum(sizes), case["q_len"], case["heads"], case["kv_heads"]
        if case["strided"]:  # q inside the fused projection's rows
            st["q"] = randn(n, t, H + 2 * kv, HD).to(dt)[:, :, :H]
        else:
            st["q"] = randn(n, t, H, HD).to(dt)
        planes = randn(2, case["groups"] * case["prefix"], kv * HD).to(dt)  # K and V planes of one decoder layer
        st["k"], st["v"] = (p.view(case["groups"], case["prefix"], kv, HD) for p in planes)
        st["prefix_lens"] = _i32(pre) if case["ragged"] else None
        st["group_start"] = _i32(np.cumsum([0] + sizes).tolist()) if case["uneven"] else None
        st["k_pages"] = st["v_pages"] = st["table"] = st["lens"] = None
        if case["suffix"]:
            st["k_pages"], st["v_pages"], st["table"] = _pages(g, suf, case["page"], kv, dt)
            st["lens"] = _i32(suf)
        return st
    if case["op"] == "kv_append":
        new, lens = _append_lens(case)
        dt, H, kv, rot = DT[case["dtype"]], case["heads"], case["kv_heads"], case["rot"]
        rows = sum(new) + case["pad"]
        fused = randn(rows, H + 2 * kv, HD).to(dt)  # the fused projection's rows
        st["q"], st["k"], st["v"] = fused[:, :H], fused[:, H:H + kv], fused[:, H + kv:]
        st["q_out"] = torch.zeros(rows, H, HD, dtype=dt, device="cuda")
        st["k_pages"], st["v_pages"], st["table"] = _pages(g, lens, case["page"], kv, dt)
        st["lens"], st["tokens"] = _i32(lens), sum(new)
        st["seq_start"] = _i32(np.cumsum([0] + new).tolist())
        st["inv_freq"] = st["positions"] = None
        if rot:
            st["inv_freq"] = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)],
                                          dtype=torch.float32, device="cuda")
            if case["far"]:  # the cache holds the end of a long stream
                at = np.concatenate([np.arange(v - m, v) for m, v in zip(new, lens)] + [np.zeros(case["pad"], int)])
                st["positions"] = _i32((at + case["far"]).tolist())
        return st
    M, N, K = case["M"], case["N"], case["K"]
    st["x"] = randn(M, K)
    st["x"].mul_(torch.exp(0.5 * randn(M, 1)))  # tokens differ in size
    st["x"] = st["x"].to(DT[case["x"]])
    st["w"] = (randn(N, K) * 32).round_().clamp_(-127, 127).to(torch.int8)
    st["w_scale"] = torch.exp(0.2 * randn(N)) * (0.02 / 32)
    st["bias"] = 0.01 * randn(N)
    st["resid"] = randn(M, N) if case["epilogue"] == RESID else None
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    if own:
        import transformer_encoder_gb300 as wenc
        if case["op"] == "prefix_attention":
            return wenc.prefix_attention(st["q"], st["k"], st["v"], prefix_lens=st["prefix_lens"],
                                         group_start=st["group_start"],
                                         max_group=case["beams"] if case["uneven"] else None, k_pages=st["k_pages"],
                                         v_pages=st["v_pages"], block_table=st["table"], lens=st["lens"])
        if case["op"] == "kv_append":
            wenc.kv_append(st["k"], st["v"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                           seq_start=st["seq_start"], q=st["q"], q_out=st["q_out"], positions=st["positions"],
                           inv_freq=st["inv_freq"], interleaved=case["interleaved"])
            return {"q": st["q_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
        xq, x_scale = wenc.quantize_rows(st["x"])
        return wenc.linear_i8(xq, x_scale, st["w"], st["w_scale"], st["bias"], epilogue=case["epilogue"],
                              resid=st["resid"])
    if case["op"] == "prefix_attention":
        return _plain_attention(st)
    if case["op"] == "kv_append":
        return _plain_append(st)
    return _plain_linear(st)


def _plain_attention(st):
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    n, t, H, _ = q.shape
    G, T, kv, _ = k.shape
    r, S, dev = H // kv, st["case"]["beams"], q.device
    seq = torch.arange(n, device=dev)
    if st["group_start"] is None:
        group, slot = seq // S, seq % S
    else:
        start = st["group_start"].long()
        group = torch.searchsorted(start[1:], seq, right=True)
        slot = seq - start[group]
    q = q.view(n, t, kv, r, HD).permute(0, 2, 1, 3, 4) * HD ** -0.5  # [n, kv, t, r, 64]
    qg = torch.zeros(G, S, kv, t, r, HD, device=dev)
    qg[group, slot] = q
    qg = qg.transpose(1, 2).reshape(G, kv, S * t * r, HD)
    s = (qg @ k.permute(0, 2, 3, 1)).view(G, kv, S, t, r, T)
    if st["prefix_lens"] is not None:
        there = torch.arange(T, device=dev) < st["prefix_lens"].view(G, 1)
        s = s.masked_fill(~there.view(G, 1, 1, 1, 1, T), -math.inf)
        v = v.masked_fill(~there.view(G, T, 1, 1), 0.0)
    s = s.transpose(1, 2)[group, slot]  # [n, kv, t, r, T]
    if st["lens"] is not None:
        at = st["table"].clamp(min=0).long()
        ks = st["k_pages"][at].flatten(1, 2).float()  # [n, L, kv, 64]
        vs = st["v_pages"][at].flatten(1, 2).float()
        L = ks.shape[1]
        j, lens = torch.arange(L, device=dev), st["lens"].long().view(n, 1)
        seen = j < (lens - t + 1 + torch.arange(t, device=dev)).unsqueeze(2)  # [n, t, L]
        vs = vs.masked_fill(~(j < lens).view(n, L, 1, 1), 0.0)
        own_s = (q.reshape(n, kv, t * r, HD) @ ks.permute(0, 2, 3, 1)).view(n, kv, t, r, L)
        s = torch.cat([s, own_s.masked_fill(~seen.view(n, 1, t, 1, L), -math.inf)], dim=4)
    m = s.amax(4, keepdim=True)
    p = torch.exp(s - m.masked_fill(m == -math.inf, 0.0))
    den = p.sum(4)
    pg = torch.zeros(G, S, kv, t, r, T, device=dev)
    pg[group, slot] = p[..., :T]
    o = (pg.transpose(1, 2).reshape(G, kv, S * t * r, T) @ v.transpose(1, 2)).view(G, kv, S, t, r, HD)
    o = o.transpose(1, 2)[group, slot]
    if st["lens"] is not None:
        o = o + (p[..., T:].reshape(n, kv, t * r, L) @ vs.transpose(1, 2)).view(n, kv, t, r, HD)
    o = o / den.masked_fill(den == 0, 1.0).unsqueeze(4)
    return o.permute(0, 2, 1, 3, 4).reshape(n, t, H, HD).to(st["q"].dtype)


def _rotated(x, positions, inv_freq, interleaved):
    if inv_freq is None:
        return x
    half = inv_freq.shape[0]
    angle = positions.double().unsqueeze(1) * inv_freq.double()
    c, s = torch.cos(angle).float().unsqueeze(1), torch.sin(angle).float().unsqueeze(1)
    f = x.float()
    if interleaved:
        a, b = f[..., 0:2 * half:2], f[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = f[..., :half], f[..., half:2 * half]
        turned = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([turned, f[..., 2 * half:]], dim=-1).to(x.dtype)


def _plain_append(st):
    n, page, dev = st["tokens"], st["case"]["page"], st["k"].device
    token, start = torch.arange(n, device=dev), st["seq_start"].long()
    seq = torch.searchsorted(start[1:], token, right=True)
    at = st["lens"].long()[seq] - (start[seq + 1] - token)
    slot = st["table"][seq, at // page].long() * page + at % page
    positions = at if st["positions"] is None else st["positions"][:n]
    kv = st["k"].shape[1]
    st["q_out"][:n] = _rotated(st["q"][:n], positions, st["inv_freq"], st["case"]["interleaved"])
    st["k_pages"].view(-1, kv, HD)[slot] = _rotated(st["k"][:n], positions, st["inv_freq"], st["case"]["interleaved"])
    st["v_pages"].view(-1, kv, HD)[slot] = st["v"][:n]
    return {"q": st["q_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _plain_linear(st):
    x = st["x"].double()
    scale = (st["x"].float().abs().amax(1) / 127.0)
    ints = torch.round(x / scale.double().unsqueeze(1)).clamp(-127, 127).float()
    y = (ints @ st["w"].float().t()) * scale.unsqueeze(1) * st["w_scale"] + st["bias"]
    if st["case"]["epilogue"] == RESID:
        return st["resid"] + y
    if st["case"]["epilogue"] == GELU:
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "prefix_attention":
        sizes, pre, suf = _attn_lens(case)
        t, H, kv, page = case["q_len"], case["heads"], case["kv_heads"], case["page"]
        q, out, at = st["q"].double(), [], 0
        for g, size in enumerate(sizes):
            kp = st["k"][g, :pre[g]].double().repeat_interleave(H // kv, 1)  # every query head with its key head
            vp = st["v"][g, :pre[g]].double().repeat_interleave(H // kv, 1)
            for s in range(at, at + size):
                k, v, own_len = kp, vp, 0
                if case["suffix"]:
                    own_len = suf[s]
                    where = torch.arange(own_len, device="cuda")
                    ids = st["table"][s].long()[where // page]
                    k = torch.cat([k, st["k_pages"][ids, where % page].double().repeat_interleave(H // kv, 1)])
                    v = torch.cat([v, st["v_pages"][ids, where % page].double().repeat_interleave(H // kv, 1)])
                for i in range(t):
                    seen = pre[g] + max(0, own_len - t + 1 + i)
                    if not seen:
                        out.append(torch.zeros(H, HD, dtype=torch.float64, device="cuda"))
                        continue
                    z = (k[:seen] * q[s, i]).sum(2) / 8.0
                    w = torch.exp(z - z.max(0).values)
                    out.append((w.unsqueeze(2) * v[:seen]).sum(0) / w.sum(0).unsqueeze(1))
            at += size
        return torch.stack(out).view(at, t, H, HD)
    if case["op"] == "kv_append":
        new, lens = _append_lens(case)
        n = sum(new)
        at = np.concatenate([np.arange(v - m, v) for m, v in zip(new, lens)]).astype(np.int64)
        seq = np.repeat(np.arange(len(new)), new)
        ids = st["table"].cpu().numpy()[seq, at // case["page"]].astype(np.int64)
        ids, slots = torch.from_numpy(ids).cuda(), torch.from_numpy(at % case["page"]).cuda()

        def turn(x):
            x = x[:n].double().clone()
            if not case["rot"]:
                return x
            pos = torch.from_numpy(at + (case["far"] if st["positions"] is not None else 0)).cuda().double()
            for i in range(case["rot"] // 2):
                a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)
                w = (pos * st["inv_freq"][i].double()).unsqueeze(1)
                xa, xb = x[:, :, a].clone(), x[:, :, b].clone()
                x[:, :, a], x[:, :, b] = xa * torch.cos(w) - xb * torch.sin(w), xa * torch.sin(w) + xb * torch.cos(w)
            return x

        q, k, v = st["q_out"].double(), st["k_pages"].double(), st["v_pages"].double()
        q[:n] = turn(st["q"])
        k[ids, slots] = turn(st["k"])
        v[ids, slots] = st["v"][:n].double()
        return {"q": q, "k_pages": k, "v_pages": v}
    x = st["x"].double()
    scale = (x.abs().max(1).values.float() / 127.0).double().unsqueeze(1)  # the scale is an fp32 number
    y = torch.round(x / scale) @ st["w"].t().double() * scale * st["w_scale"].double() + st["bias"].double()
    if case["epilogue"] == RESID:
        return y + st["resid"].double()
    if case["epilogue"] == GELU:
        return y * torch.special.ndtr(y)
    return y
