"""Tensors that the calls make belong to the stream the call runs on: with ``stream=`` given, outputs and workspaces
come from that stream's allocator, not from the current stream's, whose blocks may still be read by work queued
there, and would be handed out again while the given stream still writes them."""
import pytest

import synth
from helpers import make_encoder

pytestmark = pytest.mark.gpu


def _calls():
    import torch
    import transformer_encoder_gb300 as wenc
    r = lambda *s, t=torch.bfloat16: torch.randn(*s, device="cuda").to(t)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    f32, i8 = torch.float32, torch.int8
    q, x, w, b = r(2, 128, 4, 64), r(300, 256), r(256, 256), r(256, t=f32)
    q32, x32, w32 = q.to(f32), x.to(f32), w.to(f32)
    sa, xi, wi = torch.ones(300, device="cuda"), torch.ones(300, 256, dtype=i8, device="cuda"), torch.ones(256, 256, dtype=i8, device="cuda")
    big, bs = torch.ones(4096, 2048, dtype=i8, device="cuda"), torch.ones(4096, device="cuda")
    aq, pk = r(3, 1, 4, 64), r(1, 20, 4, 64)
    mq, mk = r(160, 1, 32, 64), r(1, 300, 32, 64)
    pages, table, lens = r(3, 8, 4, 64), i32([[0], [1], [2]]), i32([1, 2, 3])
    wl = synth.WORKLOADS["tiny_stack"]
    enc, _, _, _ = make_encoder(wl, keep_host_layers=False, max_batch=1)
    h = r(1, wl.seq_len, wl.d_model, t=f32)
    return {
        "attention": lambda **k: wenc.attention(q, q, q, **k),
        "attention_tf32": lambda **k: wenc.attention_tf32(q32, q32, q32, **k),
        "layernorm": lambda **k: wenc.layernorm(x32, b, b, **k),
        "linear": lambda **k: wenc.linear(x, w, b, **k),
        "linear_tf32": lambda **k: wenc.linear_tf32(x32, w32, b, **k),
        "encoder": lambda **k: enc.forward(h, **k),
        "quantize_rows": lambda **k: wenc.quantize_rows(x, **k),
        "linear_i8": lambda **k: wenc.linear_i8(xi, sa, wi, b, b, **k),
        "linear_i8 with a workspace": lambda **k: wenc.linear_i8(big, bs, big, bs, bs, **k),
        "prefix_attention": lambda **k: wenc.prefix_attention(aq, pk, pk, **k),
        "prefix_attention with a workspace": lambda **k: wenc.prefix_attention(mq, mk, mk, **k),
        "kv_append": lambda **k: wenc.kv_append(aq[:, 0], aq[:, 0], pages, pages.clone(), table, lens, q=aq[:, 0], **k),
    }


def test_new_tensors_come_from_the_calls_own_stream(monkeypatch):
    import torch
    calls = _calls()
    s = torch.cuda.Stream()
    want = {n: f() for n, f in calls.items()}
    torch.cuda.synchronize()
    empty, where = torch.empty, []

    def recorded(*a, **k):
        where.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **k)

    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(torch, "empty_like", lambda t: recorded(t.shape, dtype=t.dtype, device=t.device))
    here = torch.cuda.current_stream().cuda_stream
    for name, f in calls.items():
        for stream in (s, s.cuda_stream, None):
            del where[:]
            got = f(stream=stream)
            torch.cuda.synchronize()
            assert len(where) >= (2 if "workspace" in name or name == "quantize_rows" else 1), name
            assert set(where) == {here if stream is None else s.cuda_stream}, (name, stream)
            for a, b in zip(got if isinstance(got, tuple) else (got,), want[name] if isinstance(got, tuple) else (want[name],)):
                assert torch.equal(a, b), name


def test_a_block_of_the_current_stream_is_not_written_by_another():
    """Work queued on the current stream still reads a tensor that has been dropped; a call on another stream must not
    be given its block."""
    import torch
    import transformer_encoder_gb300 as wenc
    x = torch.randn(4096, 1280, device="cuda")
    ones = torch.ones(1280, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    held = torch.empty(4096, 1280, dtype=torch.bfloat16, device="cuda")
    at = held.data_ptr()
    del held
    out = wenc.layernorm(x, ones, ones, stream=s)
    assert out.data_ptr() != at
    s.synchronize()
