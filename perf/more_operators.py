"""Operators of a serving step over the paged cache, as they are measured.

- chunk_attention: chunks of new tokens (single ones, prompts, mixtures) against a paged cache, with an optional sliding
  window and first tokens that stay visible.
- kv_extend: pages, block-table entries, row offsets, positions and slots of a step's new tokens, from the lengths.
- kv_release: the pages of finished sequences, and those behind a window, back to the free ones.
- linear_i4: products with 4-bit weights that have a scale for each group of inputs.

The plain forms are elementary torch operations in 32 bits (64 for offsets).
"""
import math
import random

import numpy as np
import torch

own = False

HD = 64  # the framework's head width
GELU, RESID = 1, 2  # epilogues; 0 is the bias alone

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _attn(name, dtype, seqs, max_new, heads, kv_heads, past, page, window, sinks, mixed, ragged, pad, strided, shape):
    return dict(name=name, op="chunk_attention", dtype=dtype, seqs=seqs, max_new=max_new, heads=heads,
                kv_heads=kv_heads, past=past, page=page, window=window, sinks=sinks, mixed=mixed, ragged=ragged,
                pad=pad, strided=strided, shape=shape)


def _extend(name, seqs, max_new, past, page, ragged, pad, shape):
    return dict(name=name, op="kv_extend", seqs=seqs, max_new=max_new, past=past, page=page, ragged=ragged, pad=pad,
                shape=shape)


def _release(name, seqs, past, page, window, sinks, done, shape):
    return dict(name=name, op="kv_release", seqs=seqs, past=past, page=page, window=window, sinks=sinks, done=done,
                shape=shape)


def _i4(name, x, scale, M, N, K, group, epilogue):
    return dict(name=name, op="linear_i4", x=x, scale=scale, M=M, N=N, K=K, group=group, epilogue=epilogue)


def listed():
    return [
        # one token of one stream at the tiny dims, which sees four first tokens and a window (latency)
        _attn("stream_token_tiny", "bf16", 1, 1, 6, 6, 2000, 16, 448, 4, False, False, 0, False, 1),
        # one step of 80 long streams at the large dims, window and sinks, q a slice of the fused projection
        _attn("streams_large", "bf16", 80, 1, 20, 20, 20000, 16, 1500, 4, False, True, 0, True, 2),
        # a step of continuous batching: most of 64 requests bring one token, some a chunk of their prompt; 4 key heads
        # for 20 query heads; padding rows behind them
        _attn("mixed_step_large", "bf16", 64, 512, 20, 4, 4096, 64, 0, 0, True, True, 30, True, 3),
        # a long prompt's chunk behind what the cache holds of it
        _attn("prompt_chunk_large", "bf16", 1, 2048, 20, 4, 14000, 64, 0, 0, False, False, 0, False, 4),
        # fp32 planes (the TF32 precision), base dims: drafts and short prompts, odd pages, window and sinks
        _attn("drafts_base_f32", "f32", 24, 33, 8, 8, 2000, 24, 500, 7, False, True, 5, True, 5),
        # the next token's places of 256 requests
        _extend("extend_step", 256, 1, 2000, 16, False, 0, 6),
        # a batch of prompts and chunks: 2048 ragged requests
        _extend("extend_prompts", 2048, 500, 4000, 16, True, 100, 7),
        # requests that ended this step among 256
        _release("release_done", 256, 2000, 16, 0, 0, 0.2, 8),
        # 4096 streams: what their window has left behind since the last call, and all of those that ended
        _release("release_streams", 4096, 20000, 16, 1500, 4, 0.02, 9),
        # one token through the fused projection of the tiny dims
        _i4("qkv_one_tiny", "bf16", "f32", 1, 1152, 384, 32, 0),
        # one step of 16 windows x 5 beams through fc1 of the large dims
        _i4("fc1_beams_large", "bf16", "bf16", 80, 5120, 1280, 64, GELU),
        # ten prompts of 224 tokens through fc2 of the large dims, onto the residual stream
        _i4("fc2_prompts_large", "bf16", "bf16", 2240, 1280, 5120, 128, RESID),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _seconds(case):
    w = work(case)
    slow = 8 if case.get("dtype", case.get("x")) == "f32" else 1  # (fp32 products take several passes)
    return w["bytes"] / 6.8e12 + slow * w["flops"] / 1.9e15


def draw(rng):
    op = rng.choice(["chunk_attention", "chunk_attention", "chunk_attention", "kv_extend", "kv_release", "linear_i4",
                     "linear_i4"])
    most = max(_seconds(c) for c in listed() if c["op"] == op)
    while True:
        shape = rng.randrange(1 << 30)
        page = rng.choice([8, 16, 24, 64])
        if op == "chunk_attention":
            dtype = rng.choice(["bf16", "bf16", "f32"])
            heads, kv = rng.choice([(6, 6), (8, 8), (12, 12), (20, 20), (20, 4), (16, 2), (5, 1), (8, 4)])
            kind = rng.choice(["tokens", "mixed", "chunks", "prompt"])
            seqs = {"tokens": _log(rng, 1, 256), "mixed": _log(rng, 4, 128), "chunks": _log(rng, 2, 64),
                    "prompt": rng.randint(1, 3)}[kind]
            most_new = {"tokens": rng.choice([1, 1, 2, 4]), "mixed": _log(rng, 8, 600), "chunks": _log(rng, 2, 300),
                        "prompt": _log(rng, 64, 2048)}[kind]
            window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 16, 4000), rng.choice([0, 1, 4, 40]))])
            c = _attn(None, dtype, seqs, most_new, heads, kv, _log(rng, 1, 16000) - 1, page, window, sinks,
                      kind == "mixed", rng.random() < 0.6, rng.choice([0, 0, 1, 30]), rng.random() < 0.5, shape)
            if seqs * (c["past"] + most_new) * kv > 1 << 24:  # (the plain form's keys in 32 bits)
                continue
        elif op == "kv_extend":
            c = _extend(None, _log(rng, 1, 4096), _log(rng, 1, 2000), _log(rng, 1, 8000) - 1, page,
                        rng.random() < 0.7, rng.choice([0, 1, 100]), shape)
        elif op == "kv_release":
            window, sinks = rng.choice([(0, 0), (_log(rng, 16, 4000), rng.choice([0, 1, 4, 40]))])
            c = _release(None, _log(rng, 1, 4096), _log(rng, 1, 20000), page, window, sinks,
                         rng.choice([0.0, 0.05, 0.3, 1.0]), shape)
        else:
            group = rng.choice([32, 64, 128])
            c = _i4(None, rng.choice(["bf16", "bf16", "f32"]), rng.choice(["bf16", "f32"]), _log(rng, 1, 2240),
                    128 * _log(rng, 3, 60), 128 * _log(rng, 3, 40), group, rng.choice([0, GELU, RESID]))
        del c["name"]
        if _seconds(c) <= most:
            return c


# ------------------------------------------------------------------ what the cases' lengths are
def _chunk_lens(case):
    """(new tokens, lengths with them) of each sequence"""
    r = random.Random(case["shape"])
    n, most = case["seqs"], case["max_new"]
    if case["mixed"]:
        new = [1 if r.random() < 0.85 else r.randint(1, most) for _ in range(n)]
    else:
        new = [r.randint(0, most) if case["ragged"] and most > 1 else most for _ in range(n)]
    new[r.randrange(n)] = most
    past = [r.randint(0, case["past"]) if case["ragged"] else case["past"] for _ in range(n)]
    past[r.randrange(n)] = case["past"]
    return new, [p + m for p, m in zip(past, new)]


def _visible(case, p):
    """keys that a token at position p sees"""
    if not case["window"] or p < case["window"]:
        return p + 1
    return case["window"] + min(case["sinks"], p + 1 - case["window"])


def _extend_lens(case):
    """(new tokens, lengths before them)"""
    r = random.Random(case["shape"])
    n = case["seqs"]
    new = [r.randint(0, case["max_new"]) if case["ragged"] else case["max_new"] for _ in range(n)]
    past = [r.randint(0, case["past"]) for _ in range(n)]
    return new, past


def _release_lens(case):
    """(lengths, finished, entries given back before)"""
    r = random.Random(case["shape"])
    n, page = case["seqs"], case["page"]
    lens = [r.randint(0, case["past"]) for _ in range(n)]
    done = [r.random() < case["done"] for _ in range(n)]
    # (a call every few steps: some 40 tokens since the last)
    gone = [max(0, v - r.randint(0, 40) - case["window"] + 1) // page if case["window"] else 0 for v in lens]
    return lens, done, gone


def _gives(case, length, done, gone):
    """the ranges of table entries that a sequence gives back"""
    page = case["page"]
    first = -(-case["sinks"] // page) if case["window"] else 0
    total = -(-length // page)
    if done:
        return (0, min(first, total)), (max(first, gone), max(total, first, gone))
    end = max(0, length - case["window"] + 1) // page if case["window"] else 0
    return (0, 0), (max(first, gone), max(end, first, gone))


def work(case):
    if case["op"] == "chunk_attention":
        new, lens = _chunk_lens(case)
        e = 2 if case["dtype"] == "bf16" else 4
        H, kv = case["heads"], case["kv_heads"]
        pairs = keys = 0
        for m, v in zip(new, lens):
            if m:
                pairs += sum(_visible(case, p) for p in range(v - m, v))
                keys += _visible(dict(case, window=case["window"] + m - 1) if case["window"] else case, v - 1)
        return {"bytes": e * HD * (2 * sum(new) * H + 2 * kv * keys), "flops": 4 * HD * H * pairs}
    if case["op"] == "kv_extend":
        new, past = _extend_lens(case)
        n, page, rows = case["seqs"], case["page"], sum(new) + case["pad"]
        pages = sum(-(-(p + m) // page) + p // -page for p, m in zip(past, new))
        return {"bytes": 4 * (2 * n + 2 * pages) + 4 * (2 * n + 1) + 12 * rows, "flops": 0}
    if case["op"] == "kv_release":
        lens, done, gone = _release_lens(case)
        pages = sum(sum(b - a for a, b in _gives(case, *x)) for x in zip(lens, done, gone))
        return {"bytes": case["seqs"] * (8 + 1 + (8 if case["window"] else 0)) + 8 * pages, "flops": 0}
    M, N, K = case["M"], case["N"], case["K"]
    e, se = (2 if case["x"] == "bf16" else 4), (2 if case["scale"] == "bf16" else 4)
    out = 8 if case["epilogue"] == RESID else e
    return {"bytes": e * M * K + N * K // 2 + se * N * (K // case["group"]) + out * M * N + 4 * N, "flops": 2 * M * N * K}


# ------------------------------------------------------------------ what the program has in hand
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(g, ranges, page_total, width):
    """A table whose entries of these ranges (a list of (first, end) pairs for each sequence) name pages in shuffled
    order, -1 elsewhere, and the pages that are left."""
    there = np.zeros((len(ranges), width), dtype=bool)
    for s, spans in enumerate(ranges):
        for a, b in spans:
            there[s, a:b] = True
    order = torch.randperm(page_total, generator=g, device="cuda").to(torch.int32)
    there = torch.from_numpy(there).cuda()
    table = torch.full(there.shape, -1, dtype=torch.int32, device="cuda")
    used = int(there.sum())
    table[there] = order[:used]
    return table, order[used:]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 29)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    st = {"case": case}
    if case["op"] == "chunk_attention":
        new, lens = _chunk_lens(case)
        dt, H, kv, page = DT[case["dtype"]], case["heads"], case["kv_heads"], case["page"]
        rows = sum(new) + case["pad"]
        if case["strided"]:  # q inside the fused projection's rows
            st["q"] = randn(rows, H + 2 * kv, HD).to(dt)[:, :H]
        else:
            st["q"] = randn(rows, H, HD).to(dt)
        st["out"] = torch.zeros(rows, H, HD, dtype=dt, device="cuda")
        # the pages that a window has left behind are gone
        spans = []
        for m, v in zip(new, lens):
            total = -(-v // page)
            end = max(0, v - m - case["window"] + 1) // page if case["window"] else 0
            first = -(-case["sinks"] // page)
            spans.append([(0, min(first, total)), (end, total)] if case["window"] else [(0, total)])
        n_pages = max(1, sum(len(set(a for x in sp for a in range(*x))) for sp in spans))
        st["table"], _ = _table(g, spans, n_pages, max(1, max(-(-v // page) for v in lens)))
        st["k_pages"], st["v_pages"] = (randn(n_pages, page, kv, HD).to(dt) for _ in range(2))
        st["lens"], st["tokens"] = _i32(lens), sum(new)
        st["seq_start"] = _i32(np.cumsum([0] + new).tolist())
        return st
    if case["op"] == "kv_extend":
        new, past = _extend_lens(case)
        page, rows = case["page"], sum(new) + case["pad"]
        before = [-(-p // page) for p in past]
        after = [-(-(p + m) // page) for p, m in zip(past, new)]
        n_pages = sum(after) + 50
        st["table"], left = _table(g, [[(0, b)] for b in before], n_pages, max(1, max(after)))
        st["free_pages"] = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        st["free_pages"][:left.numel()] = left
        st["free_count"] = _i32([left.numel()])
        st["new"], st["lens"], st["rows"] = _i32(new), _i32(past), rows
        return st
    if case["op"] == "kv_release":
        lens, done, gone = _release_lens(case)
        page = case["page"]
        first = -(-case["sinks"] // page) if case["window"] else 0
        total = [-(-v // page) for v in lens]
        spans = [[(0, min(first, t)), (min(max(first, x), t), t)] for t, x in zip(total, gone)]
        n_pages = max(1, sum(total))
        st["table"], left = _table(g, spans, n_pages, max(1, max(total)))
        st["free_pages"] = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
        st["free_pages"][:left.numel()] = left
        st["free_count"] = _i32([left.numel()])
        st["lens"], st["trimmed"] = _i32(lens), _i32(gone) if case["window"] else None
        st["finished"] = torch.tensor(done, device="cuda")
        return st
    M, N, K = case["M"], case["N"], case["K"]
    st["x"] = randn(M, K)
    st["x"].mul_(torch.exp(0.5 * randn(M, 1)))  # tokens differ in size
    st["x"] = st["x"].to(DT[case["x"]])
    st["w"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    st["w_scale"] = (torch.exp(0.3 * randn(N, K // case["group"])) * (0.02 / 4)).to(DT[case["scale"]])
    st["bias"] = 0.01 * randn(N)
    st["resid"] = randn(M, N) if case["epilogue"] == RESID else None
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    case = st["case"]
    if own:
        import transformer_encoder_gb300 as wenc
        if case["op"] == "chunk_attention":
            return wenc.chunk_attention(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                                        seq_start=st["seq_start"], max_new=case["max_new"],
                                        window=case["window"] or None, sinks=case["sinks"], out=st["out"])
        if case["op"] == "kv_extend":
            lens, count, start, positions, slots = wenc.kv_extend(st["new"], st["lens"], st["table"], st["free_pages"],
                                                                  st["free_count"], case["page"], st["rows"])
            return {"table": st["table"], "lens": lens, "count": count, "seq_start": start, "positions": positions,
                    "slots": slots}
        if case["op"] == "kv_release":
            lens, count, trimmed = wenc.kv_release(st["lens"], st["table"], st["free_pages"], st["free_count"],
                                                   case["page"], finished=st["finished"],
                                                   window=case["window"] or None, sinks=case["sinks"],
                                                   trimmed=st["trimmed"])
            return {"free_pages": st["free_pages"], "lens": lens, "count": count, "trimmed": trimmed}
        return wenc.linear_i4(st["x"], st["w"], st["w_scale"], st["bias"], epilogue=case["epilogue"],
                              resid=st["resid"])
    if case["op"] == "chunk_attention":
        return _plain_attention(st)
    if case["op"] == "kv_extend":
        return _plain_extend(st)
    if case["op"] == "kv_release":
        return _plain_release(st)
    return _plain_linear(st)


def _plain_attention(st):
    """Sequences in batches of padded rows, each against the positions that its first and last token span."""
    case, dev = st["case"], st["q"].device
    new, lens = _chunk_lens(case)
    H, kv, page, W, S = case["heads"], case["kv_heads"], case["page"], case["window"], case["sinks"]
    r, n = H // kv, len(new)
    start = np.cumsum([0] + new)
    by_size = sorted((s for s in range(n) if new[s]), key=lambda s: (new[s], lens[s]))
    at = 0
    while at < len(by_size):
        batch, t, L = [], 0, 0
        while at < len(by_size):  # as many as keep the scores within 2^29 numbers
            s = by_size[at]
            t2, L2 = new[s], max(L, S + min(W + new[s] - 1, lens[s]) if W else lens[s])
            if batch and (len(batch) + 1) * H * t2 * L2 > 1 << 29:
                break
            batch.append(s)
            t, L, at = t2, L2, at + 1
        b = len(batch)
        ids = torch.tensor(batch, device=dev)
        m = torch.tensor([new[s] for s in batch], device=dev).view(b, 1)
        end = torch.tensor([lens[s] for s in batch], device=dev).view(b, 1)
        first = torch.tensor([int(start[s]) for s in batch], device=dev).view(b, 1)
        i = torch.arange(t, device=dev)
        rows = (first + torch.minimum(i, m - 1))  # [b, t], the last row again behind a chunk's end
        pos = (end - m + torch.minimum(i, m - 1)).unsqueeze(2)  # [b, t, 1]
        j = torch.arange(L, device=dev).view(1, L)
        if W:  # the sinks, then the positions from the first token's window on
            low = (end - m - W + 1).clamp(min=S)
            j = torch.where(j < S, j, low + j - S)
        there = (j < end).expand(b, L)
        j = torch.minimum(j, end - 1)
        pages = st["table"][ids.view(b, 1), j // page].long()
        there = there & (pages >= 0)
        slot = pages.clamp(min=0) * page + j % page
        ks = st["k_pages"].view(-1, kv, HD)[slot].float()  # [b, L, kv, 64]
        vs = st["v_pages"].view(-1, kv, HD)[slot].float().masked_fill(~there.view(b, L, 1, 1), 0.0)
        seen = there.unsqueeze(1) & (j.unsqueeze(1) <= pos)
        if W:
            seen = seen & ((j.unsqueeze(1) > pos - W) | (j.unsqueeze(1) < S))
        q = st["q"][rows].float().view(b, t, kv, r, HD).permute(0, 2, 3, 1, 4).reshape(b, kv, r * t, HD) * HD ** -0.5
        s = (q @ ks.permute(0, 2, 3, 1)).view(b, kv, r, t, L)
        s = s.masked_fill(~seen.view(b, 1, 1, t, L), -math.inf)
        p = torch.exp(s - s.amax(4, keepdim=True))
        den = p.sum(4, keepdim=True)
        o = (p.view(b, kv, r * t, L) @ vs.transpose(1, 2)).view(b, kv, r, t, HD) / den
        o = o.permute(0, 3, 1, 2, 4).reshape(b * t, H, HD).to(st["q"].dtype)
        st["out"][rows.flatten()] = o
    return st["out"]


def _plain_extend(st):
    page, rows = st["case"]["page"], st["rows"]
    new, lens, dev = st["new"].long(), st["lens"].long(), st["new"].device
    n = new.numel()
    start = torch.zeros(n + 1, dtype=torch.long, device=dev)
    start[1:] = new.cumsum(0)
    before = (lens + page - 1) // page
    need = (lens + new + page - 1) // page - before
    base = need.cumsum(0) - need
    col = torch.arange(st["table"].shape[1], device=dev)
    entry = col - before.view(n, 1)  # which of a sequence's new pages a table entry is
    fresh = (entry >= 0) & (entry < need.view(n, 1))
    at = st["free_count"].long() - 1 - (base.view(n, 1) + entry)
    st["table"].copy_(torch.where(fresh, st["free_pages"][at.clamp(0, st["free_pages"].numel() - 1)], st["table"]))
    row = torch.arange(rows, device=dev)
    seq = torch.searchsorted(start[1:], row, right=True)
    real = seq < n
    seq = seq.clamp(max=n - 1)
    pos = torch.where(real, lens[seq] + row - start[seq], 0)
    slots = torch.where(real, st["table"][seq, pos // page].long() * page + pos % page, -1)
    return {"table": st["table"], "lens": (lens + new).int(), "count": st["free_count"] - need.sum().int(),
            "seq_start": start.int(), "positions": pos.int(), "slots": slots}


def _plain_release(st):
    case, page = st["case"], st["case"]["page"]
    lens, done, dev = st["lens"].long(), st["finished"], st["lens"].device
    n, zero = lens.numel(), torch.zeros_like(st["lens"], dtype=torch.long)
    total = (lens + page - 1) // page
    first = -(-case["sinks"] // page) if case["window"] else 0
    gone = st["trimmed"].long() if case["window"] else zero
    low = gone.clamp(min=first)
    end = (lens - case["window"] + 1).clamp(min=0) // page if case["window"] else zero
    col = torch.arange(st["table"].shape[1], device=dev).view(1, -1)
    back = (col >= low.view(n, 1)) & (col < torch.where(done, total, end).view(n, 1))
    back = back | (done.view(n, 1) & (col < total.clamp(max=first).view(n, 1)))
    flat = back.flatten()
    order = flat.long().cumsum(0) - 1 + st["free_count"]
    # (the entries that stay are written behind the array's end, and cut off)
    cap = st["free_pages"].numel()
    room = torch.cat([st["free_pages"], st["free_pages"].new_zeros(1)])
    room[torch.where(flat, order, cap)] = st["table"].flatten()
    st["free_pages"].copy_(room[:cap])
    trimmed = torch.where(done, zero, torch.maximum(gone, end)).int() if case["window"] else None
    return {"free_pages": st["free_pages"], "lens": torch.where(done, zero, lens).int(),
            "count": st["free_count"] + flat.sum().int(), "trimmed": trimmed}


def _plain_linear(st):
    case = st["case"]
    u = torch.stack([st["w"] & 15, st["w"] >> 4], dim=2).flatten(1)  # the low half of a byte comes first
    w = (u.float() - 8.0) * st["w_scale"].float().repeat_interleave(case["group"], 1)
    y = st["x"].float() @ w.t() + st["bias"]
    if case["epilogue"] == RESID:
        return st["resid"] + y
    if case["epilogue"] == GELU:
        y = 0.5 * y * torch.erfc(-y * math.sqrt(0.5))
    return y.to(st["x"].dtype)


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    if work(case)["flops"] > 1.0e13 or (case["op"] == "chunk_attention" and work(case)["flops"] > 6.0e10):
        return None
    st = prepare(case, seed)
    if case["op"] == "chunk_attention":
        new, lens = _chunk_lens(case)
        H, kv, page = case["heads"], case["kv_heads"], case["page"]
        out, row = st["out"].double(), 0
        for s, (m, v) in enumerate(zip(new, lens)):
            if not m:
                continue
            p = np.arange(v - m, v)[:, None]
            j = np.arange(v)[None]
            seen = j <= p
            if case["window"]:
                seen &= (j > p - case["window"]) | (j < case["sinks"])
            keys = np.flatnonzero(seen.any(0))
            hide = torch.from_numpy(~seen[:, keys]).cuda()
            where = torch.from_numpy(keys).cuda()
            ids = st["table"][s].long()[where // page]
            k, v64 = (x[ids, where % page].double() for x in (st["k_pages"], st["v_pages"]))
            for h in range(H):
                z = (st["q"][row:row + m, h].double() @ k[:, h // (H // kv)].t()) / 8.0
                z[hide] = -math.inf
                out[row:row + m, h] = torch.softmax(z, 1) @ v64[:, h // (H // kv)]
            row += m
        return out
    if case["op"] == "kv_extend":
        new, past = _extend_lens(case)
        page = case["page"]
        table, free = st["table"].cpu().numpy(), st["free_pages"].cpu().numpy()
        count = int(st["free_count"])
        positions, slots = [], []
        for s, (m, p) in enumerate(zip(new, past)):
            for e in range(-(-p // page), -(-(p + m) // page)):
                count -= 1
                table[s, e] = free[count]
            at = np.arange(p, p + m)
            positions.append(at)
            slots.append(table[s, at // page].astype(np.int64) * page + at % page)
        positions.append(np.zeros(case["pad"], np.int64))
        slots.append(np.full(case["pad"], -1, np.int64))
        return {"table": torch.from_numpy(table).cuda(), "lens": _i32([a + b for a, b in zip(new, past)]),
                "count": _i32([count]), "seq_start": _i32(np.cumsum([0] + new).tolist()),
                "positions": _i32(np.concatenate(positions).tolist()),
                "slots": torch.from_numpy(np.concatenate(slots)).cuda()}
    if case["op"] == "kv_release":
        lens, done, gone = _release_lens(case)
        table, free = st["table"].cpu().numpy(), st["free_pages"].cpu().numpy()
        count, marks = int(st["free_count"]), []
        for s, x in enumerate(zip(lens, done, gone)):
            spans = _gives(case, *x)
            for a, b in spans:
                free[count:count + b - a] = table[s, a:b]
                count += b - a
            end = max(0, lens[s] - case["window"] + 1) // case["page"]
            marks.append(0 if done[s] else max(gone[s], end))
        return {"free_pages": torch.from_numpy(free).cuda(), "lens": _i32([0 if d else v for v, d in zip(lens, done)]),
                "count": _i32([count]), "trimmed": _i32(marks) if case["window"] else None}
    x, group = st["x"].double(), case["group"]
    y = st["bias"].double().expand(case["M"], case["N"]).clone()
    ints = torch.empty(case["N"], case["K"], dtype=torch.float64, device="cuda")
    ints[:, 0::2], ints[:, 1::2] = (st["w"] & 15).double() - 8.0, (st["w"] >> 4).double() - 8.0
    for i in range(case["K"] // group):
        k = slice(i * group, (i + 1) * group)
        y += (x[:, k] @ ints[:, k].t()) * st["w_scale"][:, i].double()
    if case["epilogue"] == RESID:
        return y + st["resid"].double()
    if case["epilogue"] == GELU:
        return y * torch.special.ndtr(y)
    return y
