"""wenc_prefix_attention in the form that joins partial results (many rows per key head): what a row gives does not
depend on how many rows it shares its prefix with.

The bound is that of the one-launch form for both types (the derivation is in test_gpu_prefix_attention.py): for bf16
  |err| <= 2^-8 |o| + (2 e + 2^-16 + 2 n 2^-23) sum_j p_j |v_j|,  e = 1.1 d + 2^-16 + 2^-21,
with 2^-16 for two-part probabilities. Of some 10^5 elements hundreds are so near zero that the last term is most of
their bound; probabilities held in one bf16 number (2^-9 each, over the square root of the keys) pass it there.
"""
import numpy as np
import pytest

from oracle import decode
from test_gpu_prefix_attention import Case, _joins

pytestmark = pytest.mark.gpu


def _check_two_parts(c, out):
    got = out.double().cpu().numpy()
    ref, absv, A = decode.prefix_attention(c.q.astype(np.float64), c.prefixes, c.owns, c.groups, 0.125)
    keys = max(p[0].shape[0] for p in c.prefixes) + max(o[0].shape[0] for o in c.owns)
    e = 2.0 ** -16 + 2.0 ** -21 + 1.1 * A[..., None] * 0.125 * 64 * 2.0 ** -23
    bound = 2.0 ** -8 * np.abs(ref) + (2 * e + 2.0 ** -16 + 2 * keys * 2.0 ** -23) * absv
    assert np.isfinite(got).all()
    worst = float((np.abs(got - ref) / bound).max())
    assert worst <= 1, f"{worst:.2f} x the bound"


@pytest.mark.parametrize("H,Hkv,q_len,sizes,pre", [
    (32, 32, 1, [160], [129]), (96, 32, 1, [60, 5], [257, 40]), (40, 1, 1, [130, 2], [300, 64]), (4, 4, 7, [40, 180], [500, 127]),
    (1, 1, 1, [2500], [1700])])
def test_probabilities_keep_two_parts_with_many_rows(H, Hkv, q_len, sizes, pre):
    """(with one-part probabilities the first four reached 3.4 to 5.2 times this bound)"""
    c = Case("bf16", sizes, q_len, H, Hkv, pre, None, uneven=len(sizes) > 1, seed=H + q_len, prefix_max=max(pre) + 37)
    assert _joins(c)
    _check_two_parts(c, c.run())


@pytest.mark.parametrize("dtype,H,Hkv,n,T", [("bf16", 32, 32, 160, 300), ("f32", 32, 32, 245, 100), ("bf16", 130, 1, 300, 300)])
def test_append_and_joined_attention_back_to_back(dtype, H, Hkv, n, T):
    """Steps of an append and the joined form in one stream, nothing waiting between them, with new keys, lengths,
    tables and queries in the same buffers each time: the same bits as with a synchronisation after every call, eager
    and captured. (The own keys' kernel reads what the append two launches before it wrote.)"""
    import torch
    from transformer_encoder_gb300 import kv_append, prefix_attention, sync_status
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)
    PAGE, WIDTH, STEPS = 8, 4, 6
    kp, vp = rnd(1, T, Hkv, 64), rnd(1, T, Hkv, 64)
    feeds = [dict(q=rnd(n, 1, H, 64), k=rnd(9 * n, Hkv, 64), v=rnd(9 * n, Hkv, 64),
                  lens=torch.randint(9, PAGE * WIDTH + 1, (n,), generator=g, device="cuda", dtype=torch.int32),
                  table=torch.randperm(n * WIDTH, generator=g, device="cuda").to(torch.int32).view(n, WIDTH))
             for _ in range(STEPS)]
    live = {k: torch.zeros_like(t) for k, t in feeds[0].items()}
    pages = torch.zeros(2, n * WIDTH, PAGE, Hkv, 64, dtype=dt, device="cuda")

    def append_and_attend():  # nine new tokens a sequence, then the newest of them attends
        kv_append(live["k"], live["v"], pages[0], pages[1], live["table"], live["lens"])
        return prefix_attention(live["q"], kp, vp, k_pages=pages[0], v_pages=pages[1], block_table=live["table"],
                                lens=live["lens"])

    def steps(once, wait):
        pages.zero_()
        outs = []
        for f in feeds:
            for k, t in f.items():
                live[k].copy_(t)
            if wait:
                torch.cuda.synchronize()
            outs.append(once().clone())
            if wait:
                torch.cuda.synchronize()
        sync_status()
        return outs

    def apart():
        kv_append(live["k"], live["v"], pages[0], pages[1], live["table"], live["lens"])
        torch.cuda.synchronize()
        return prefix_attention(live["q"], kp, vp, k_pages=pages[0], v_pages=pages[1], block_table=live["table"],
                                lens=live["lens"])

    want = steps(apart, True)
    assert not torch.equal(want[0], want[1])
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(steps(append_and_attend, False), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = append_and_attend()

    def replay():
        graph.replay()
        return out

    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(steps(replay, False), want))


def _room(c):
    """Bytes of workspace the case needs, exactly."""
    import re
    import torch
    from transformer_encoder_gb300 import WencError, prefix_attention
    with pytest.raises(WencError) as e:
        prefix_attention(c.tq, **c.kw, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    return int(re.search(r"workspace of (\d+) bytes needed", str(e.value)).group(1))


@pytest.mark.parametrize("dtype,H,Hkv,sizes,pre", [
    ("bf16", 32, 32, [160, 90], [700, 0]), ("bf16", 130, 1, [300], [300]), ("f32", 32, 32, [245, 60], [0, 200]),
    ("f32", 130, 1, [50, 44], [150, 3])])
def test_a_given_workspace_may_hold_anything(dtype, H, Hkv, sizes, pre):
    """Many slots of the partial results stay unwritten (short and empty prefixes and own lists): what their memory held,
    NaN or the call's before, is not in the result; and two such calls at once, each with its own, give the same bits."""
    import torch
    from transformer_encoder_gb300 import prefix_attention, sync_status
    r = np.random.default_rng(H + sizes[0])
    cases = [Case(dtype, sizes, 1, H, Hkv, pre, [int(x) for x in r.integers(0, 40, sum(sizes)) * r.integers(0, 2, sum(sizes))],
                  page=8, uneven=len(sizes) > 1, seed=s, prefix_max=900) for s in (34, 35)]
    assert all(_joins(c) for c in cases)
    want = [c.run() for c in cases]
    cases[0].check(want[0])
    guard = 4096
    rooms = [torch.full((_room(c) + guard,), 255, dtype=torch.uint8, device="cuda") for c in cases]
    for _ in range(3):  # NaN in every slot, then what the last call left
        assert torch.equal(cases[0].run(workspace=rooms[0][:-guard]), want[0])
    assert torch.equal(cases[1].run(workspace=rooms[0][:_room(cases[1])]), want[1])  # another call's partial results
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for c, s, w, o in zip(cases, streams, rooms, outs):
            prefix_attention(c.tq, **c.kw, out=o, workspace=w[:-guard], stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    sync_status()
    assert all((w[-guard:] == 255).all() for w in rooms)
