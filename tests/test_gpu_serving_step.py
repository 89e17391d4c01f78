"""A serving loop of the operators together: pages planned from lengths, projections in 4 bits, keys and values appended, chunks
attended, pages given back. Prompts, drafts, single tokens and sequences that end mix in one batch; a plain cache on the host, which
keeps every sequence's keys and values in order, says what each step has to give.

Bounds: a step's queries, keys and values come from the operator itself (its own test holds it to its definition), so the
attention is compared on them: bf16 output, 2^-8 of the value for the rounding and 2^-8 of the largest value of V's weighted
magnitudes, which stay below 4, times what the probabilities' arithmetic leaves (2^-13 for these few hundred keys)."""
import numpy as np
import pytest

from test_gpu_chunk_attention import plain

pytestmark = pytest.mark.gpu

D, H, HKV, PAGE, WINDOW, SINKS = 256, 4, 2, 8, 40, 4


class Model:
    def __init__(self, window, seed):
        import torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.window, self.sinks = window, SINKS if window else 0
        rows = (H + 2 * HKV) * 64
        self.wqkv = torch.randint(0, 256, (rows, D // 2), generator=g, device="cuda", dtype=torch.uint8)
        self.wo = torch.randint(0, 256, (D, H * 32), generator=g, device="cuda", dtype=torch.uint8)
        self.sqkv = torch.rand(rows, D // 32, generator=g, device="cuda") * 0.02
        self.so = (torch.rand(D, H * 64 // 64, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
        self.b, self.bo = torch.randn(rows, generator=g, device="cuda") * 0.1, torch.randn(D, generator=g, device="cuda") * 0.1
        self.inv_freq = 10000.0 ** (-torch.arange(32, device="cuda", dtype=torch.float32) / 32)


class Pool:
    def __init__(self, n_seqs, n_pages, width):
        import torch
        self.k, self.v = (torch.full((n_pages, PAGE, HKV, 64), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
        self.table = torch.full((n_seqs, width), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(n_pages, device="cuda").to(torch.int32)
        self.count = torch.tensor([n_pages], dtype=torch.int32, device="cuda")
        self.lens, self.trimmed = (torch.zeros(n_seqs, dtype=torch.int32, device="cuda") for _ in range(2))


def step(m, pool, x, stream, new, finished, max_new):
    """One step as a program runs it; everything it needs lives on the device. (lens and count pass to and fro between two
    buffers, so that a captured step can be replayed.)"""
    from transformer_encoder_gb300 import EPI_BIAS_RESID_F32, chunk_attention, kv_append, kv_extend, kv_release, linear_i4
    rows = x.shape[0]
    lens, count, start, positions, _ = kv_extend(new, pool.lens, pool.table, pool.free, pool.count, PAGE, rows)
    qkv = linear_i4(x, m.wqkv, m.sqkv, m.b).view(rows, H + 2 * HKV, 64)
    q = kv_append(qkv[:, H:H + HKV], qkv[:, H + HKV:], pool.k, pool.v, pool.table, lens, seq_start=start, q=qkv[:, :H],
                  positions=positions, inv_freq=m.inv_freq)
    o = chunk_attention(q, pool.k, pool.v, pool.table, lens, seq_start=start, max_new=max_new, window=m.window, sinks=m.sinks)
    linear_i4(o.view(rows, H * 64), m.wo, m.so, m.bo, EPI_BIAS_RESID_F32, resid=stream, out=stream)
    kv_release(lens, pool.table, pool.free, count, PAGE, finished=finished, window=m.window, sinks=m.sinks,
               trimmed=pool.trimmed if m.window else None, lens_out=pool.lens, free_count_out=pool.count,
               **(dict(trimmed_out=m.marks) if m.window else {}))
    if m.window:
        pool.trimmed.copy_(m.marks)
    return q, qkv, o


@pytest.mark.parametrize("window", [None, WINDOW])
@pytest.mark.parametrize("captured", [False, True])
def test_a_loop_of_steps(window, captured):
    import torch
    from transformer_encoder_gb300 import kv_append, sync_status
    r = np.random.default_rng(3)
    n, rows, steps, max_new = 9, 330, 7, 150
    m, pool = Model(window, 5), Pool(n, 400, 900)
    m.marks = torch.zeros(n, dtype=torch.int32, device="cuda")
    x, stream = torch.zeros(rows, D, device="cuda", dtype=torch.bfloat16), torch.zeros(rows, D, device="cuda")
    new, finished = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.bool, device="cuda")
    graph = None
    if captured:  # (a step of no tokens warms up, and is what is captured)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(m, pool, x, stream, new, finished, max_new)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q, qkv, o = step(m, pool, x, stream, new, finished, max_new)
    cache = [(torch.zeros(0, HKV, 64, device="cuda"), torch.zeros(0, HKV, 64, device="cuda")) for _ in range(n)]
    for it in range(steps):
        counts = [int(r.choice([0, 1, 1, 2, 17])) for _ in range(n)]
        counts[it % n] = 150 if it % 2 == 0 else 33  # a prompt, or a part of one
        done = [bool(r.random() < 0.15) and it > 1 for _ in range(n)]
        total = sum(counts)
        new.copy_(torch.tensor(counts, dtype=torch.int32))
        finished.copy_(torch.tensor(done))
        x.copy_(torch.randn(rows, D, device="cuda"))
        stream.copy_(torch.randn(rows, D, device="cuda"))
        before = stream.clone()
        held = [int(v) for v in pool.lens]
        if captured:
            graph.replay()
        else:
            q, qkv, o = step(m, pool, x, stream, new, finished, max_new)
        sync_status()
        # the keys as they stand in the cache: turned by their positions (by kv_append into pages of its own)
        pages = torch.zeros(2, -(-rows // 1), 1, HKV, 64, device="cuda", dtype=torch.bfloat16)
        start = np.cumsum([0] + counts)
        positions = torch.tensor([h + i for h, c in zip(held, counts) for i in range(c)] + [0] * (rows - total), dtype=torch.int32, device="cuda")
        every = torch.arange(rows, dtype=torch.int32, device="cuda").view(rows, 1)
        kv_append(qkv[:, H:H + HKV], qkv[:, H + HKV:], pages[0], pages[1], every, torch.ones(rows, dtype=torch.int32, device="cuda"),
                  positions=positions, inv_freq=m.inv_freq)
        want, magnitude = torch.zeros(total, H, 64, dtype=torch.float64, device="cuda"), torch.zeros(total, H, 64, dtype=torch.float64, device="cuda")
        for s, c in enumerate(counts):
            a, b = int(start[s]), int(start[s + 1])
            cache[s] = tuple(torch.cat([old, pages[i, a:b, 0].float()]) for i, old in enumerate(cache[s]))
            if c:
                k, v = (t.double() for t in cache[s])
                want[a:b], magnitude[a:b], _ = plain(q[a:b].double(), k, v, torch.arange(k.shape[0] - c, k.shape[0], device="cuda"),
                                                     window or 0, m.sinks, 0.125)
            if done[s]:
                cache[s] = tuple(t[:0] for t in cache[s])
        err = (o[:total].double() - want).abs()
        assert (err <= 2.0 ** -8 * want.abs() + 2.0 ** -13 * magnitude).all(), it
        assert (o[total:] == 0).all()
        # lengths, and pages: each is free, or some sequence's, once
        assert [int(v) for v in pool.lens] == [t[0].shape[0] for t in cache]
        table, free, count = pool.table.cpu().numpy(), pool.free.cpu().numpy(), int(pool.count)
        marks = pool.trimmed.tolist()
        first = -(-m.sinks // PAGE)
        owned = [int(table[s, e]) for s in range(n) for e in range(-(-int(pool.lens[s]) // PAGE)) if e < first or e >= marks[s]]
        assert sorted(owned + free[:count].tolist()) == list(range(400)), it
        if window:
            assert all(mk == max(0, int(v) - window + 1) // PAGE for mk, v in zip(marks, pool.lens))
        # what is left of the stream: the residual, with the projection of zeros (the bias) on padding rows
        assert torch.equal(stream[total:], before[total:] + m.bo)


def test_two_calls_at_once_have_a_workspace_each():
    """Long chunks on two streams at the same time: both right, with workspaces of their own."""
    import torch
    from test_gpu_chunk_attention import Case
    from transformer_encoder_gb300 import chunk_attention, sync_status
    a, b = Case("bf16", [600, 1], [900, 50], 8, 2, seed=21, wide=True), Case("bf16", [40, 700], [3, 1500], 8, 2, 300, 4, seed=22, wide=True)
    want = [c.run() for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [[torch.zeros_like(w) for _ in range(6)] for w in want]
    for i in range(6):
        for c, s, o in zip((a, b), streams, outs):
            with torch.cuda.stream(s):
                chunk_attention(c.q, c.kc, c.vc, c.table, c.tlens, seq_start=c.tstart, max_new=max(c.new), window=c.window or None,
                                sinks=c.sinks, out=o[i])
    torch.cuda.synchronize()
    sync_status()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, w) for x in o)
