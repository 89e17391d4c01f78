"""The index-checked build on the decode-side operators: every form of the shared-prefix attention, the append, the 8-bit rows and
their products run with every index check live, at ragged sizes; the device error word stays clear and every output is
bit-equal to the normal build's. Each build runs in a process of its own."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu

CHILD = r"""
import hashlib, json, sys
import numpy as np
import torch
sys.path.insert(0, %(root)r)
sys.path.insert(0, %(root)r + "/tests")
import transformer_encoder_gb300 as w
from test_gpu_prefix_attention import Case as Attention, _joins
from test_gpu_kv_append import Case as Append
assert w.lib_path.endswith(%(lib)r), w.lib_path
res = {}

def add(name, *tensors):
    w.sync_status()
    res[name] = hashlib.sha256(b"".join(t.contiguous().view(torch.uint8).cpu().numpy().tobytes() for t in tensors)).hexdigest()

r = np.random.default_rng(3)
own = lambda n, most: [int(x) for x in r.integers(0, most, n)]
forms = [  # dtype, group sizes, q_len, H, Hkv, prefixes, own lengths, page, joins
    ("bf16", [5], 1, 6, 6, [1500], None, 16, False), ("f32", [5], 1, 6, 6, [700], None, 16, False),
    ("bf16", [1, 4, 2], 3, 20, 4, [40, 0, 129], own(7, 90), 24, False), ("f32", [1, 4, 2], 3, 20, 4, [40, 0, 129], own(7, 90), 24, False),
    ("bf16", [1, 1, 1], 1, 4, 2, None, [257, 0, 31], 3, False), ("f32", [1, 1], 8, 5, 1, None, [9, 130], 1, False),
    ("bf16", [160, 5], 1, 32, 32, [257, 129], own(165, 40), 8, True), ("f32", [245], 1, 32, 32, [100], own(245, 30), 8, True),
    ("bf16", [40, 180], 7, 4, 4, [500, 127], own(220, 60), 16, True), ("bf16", [300], 1, 130, 1, [300], own(300, 20), 8, True),
    ("f32", [50], 1, 130, 1, [150], own(50, 20), 8, True), ("f32", [1200], 1, 8, 8, [65], None, 8, True),
    ("bf16", [1] * 5, 130, 40, 20, None, [200, 130, 64, 0, 131], 24, True), ("f32", [3, 2], 130, 40, 20, [300, 65], [200, 130, 64, 0, 131], 24, True)]
for i, (dtype, sizes, q_len, H, Hkv, pre, suf, page, joins) in enumerate(forms):
    for bad in (False, True):
        c = Attention(dtype, sizes, q_len, H, Hkv, pre, suf, page=page, uneven=pre is not None and len(sizes) > 1, seed=i, strided=i %% 2 == 1)
        assert _joins(c) == joins, i
        if bad:  # values that are no numbers take the rows' second way
            (c.kw["v_prefix"] if pre else c.kw["v_pages"])[0, 0, 0, 3] = float("inf")
        add(f"attention_{i}_{bad}", torch.nan_to_num(c.run().float(), 9.0, 8.0, 7.0))
for i, (dtype, new, H, Hkv, rot, inter, page) in enumerate([
        ("bf16", [1], 6, 6, 64, False, 16), ("f32", [1] * 80, 8, 8, 32, True, 24), ("bf16", own(16, 300), 20, 4, 64, False, 64),
        ("f32", own(9, 50), 5, 1, 16, False, 1), ("bf16", own(40, 33), 16, 2, 0, False, 3)]):
    c = Append(dtype, new, own(len(new), 40), H, Hkv, rot, interleaved=inter, page=page, pad=3, seed=i)
    out = c.run()
    add(f"append_{i}", c.kc, c.vc, *([] if out is None else [out]))
for rows, d in ((1, 16), (5, 64), (3, 1040), (33, 5120), (2, 40000), (2, 80000)):
    for t in (torch.bfloat16, torch.float32):
        x = torch.from_numpy(r.standard_normal((rows, d)).astype(np.float32)).cuda().to(t)
        add(f"rows_{rows}_{d}_{t}", *w.quantize_rows(x))
for M, N, K in ((1, 128, 64), (1, 1536, 384), (8, 5120, 1280), (16, 256, 6400), (17, 128, 64), (80, 5120, 1280), (129, 384, 1024),
                (300, 1280, 5120), (1500, 1536, 512), (700, 4096, 192)):
    a, b = (torch.from_numpy(r.integers(-127, 128, s).astype(np.int8)).cuda() for s in ((M, K), (N, K)))
    sa, sb, bias = (torch.from_numpy(r.random(n).astype(np.float32)).cuda() for n in (M, N, N))
    resid = torch.from_numpy(r.standard_normal((M, N)).astype(np.float32)).cuda()
    for epi in (0, 1, 2):
        add(f"linear_i8_{M}_{N}_{K}_{epi}", w.linear_i8(a, sa, b, sb * 1e-4, bias, epi, resid=resid))
print(json.dumps(res))
"""


def _run(lib):
    r = subprocess.run([sys.executable, "-c", CHILD % {"root": ROOT, "lib": lib}], capture_output=True, text=True,
                       env=dict(os.environ, WENC_LIBRARY=lib), timeout=900)
    assert r.returncode == 0, r.stderr[-3000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_index_checked_build_runs_clean_and_bit_equal():
    from transformer_encoder_gb300.build import build
    build()
    build(bounds_check=True)
    normal = _run("libwenc.so")
    checked = _run("libwenc_bounds.so")
    assert normal.keys() == checked.keys() and len(normal) > 70
    for k in normal:
        assert normal[k] == checked[k], k
