"""The index-checked build on the chunk attention, the page plans and the 4-bit product: every form runs with every index check live, at
ragged sizes; the device error word stays clear and every output is bit-equal to the normal build's. Each build runs in a
process of its own."""
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
from test_gpu_chunk_attention import Case as Chunk
from test_gpu_linear_i4 import Case as Linear
from test_gpu_pages import Cache, _extend, _t
assert w.lib_path.endswith(%(lib)r), w.lib_path
res = {}

def add(name, *tensors):
    w.sync_status()
    res[name] = hashlib.sha256(b"".join(t.contiguous().view(torch.uint8).cpu().numpy().tobytes() for t in tensors)).hexdigest()

r = np.random.default_rng(3)
ints = lambda n, most: [int(x) for x in r.integers(0, most, n)]
for i, (new, past, H, kv, window, sinks, page, pad) in enumerate([
        ([1], [2000], 6, 6, 448, 4, 16, 0), ([1, 0, 1], [16, 5, 300], 4, 2, 0, 0, 1, 2), ([1, 0, 2, 130, 1, 33, 257], ints(7, 300), 20, 4, 0, 0, 24, 9),
        ([700, 1, 40], [2500, 0, 100], 6, 2, 333, 5, 8, 0), ([300], [0], 40, 1, 0, 0, 3, 1), ([64] * 5, ints(5, 2000), 8, 8, 0, 0, 64, 0),
        ([1] * 40, ints(40, 900), 16, 2, 100, 40, 16, 0), ([500] * 3, ints(3, 50), 130, 1, 0, 0, 16, 3)]):
    for dtype in ("bf16", "f32"):
        for bad in (False, True):
            c = Chunk(dtype, new, past, H, kv, window, sinks, page=page, pad=pad, strided=i %% 2 == 1, seed=i, odd_pages=i %% 3 == 2, wide=dtype == 'bf16' and max(new) > 60)
            if bad:  # values that are no numbers take the rows' second way
                c.vc[int(c.table[len(new) - 1][(c.lens[-1] - 1) // page]), (c.lens[-1] - 1) %% page, 0, 3] = float("inf")
            add(f"chunk_{i}_{dtype}_{bad}", torch.nan_to_num(c.run().float(), 9.0, 8.0, 7.0))
for i, (n, most, past, page, pad) in enumerate([(1, 1, 0, 16, 0), (256, 1, 500, 16, 3), (33, 600, 50, 24, 3), (2049, 20, 100, 64, 1), (9000, 1, 4, 3, 0)]):
    new, lens = r.integers(0, most + 1, n).tolist(), r.integers(0, past + 1, n).tolist()
    c = Cache(lens, page, -(-(most + past) // page) + 2, sum(-(-m // page) + 1 for m in new) + 2, n)
    table, out = _extend(c, new, sum(new) + pad)
    add(f"extend_{i}", table, *out)
    free = torch.from_numpy(c.free).cuda()
    done = torch.from_numpy(r.random(n) < 0.3).cuda()
    add(f"release_{i}", *w.kv_release(_t(lens), table, free, _t([c.count]), page, finished=done, window=37, sinks=5, trimmed=_t([0] * n)), free)
for M, N, K, group in ((1, 1152, 384, 32), (7, 128, 128, 128), (16, 256, 8064, 64), (17, 128, 128, 32), (80, 5120, 1280, 64), (129, 384, 1024, 128),
                       (700, 256, 1280, 32), (2240, 1280, 640, 64)):
    for x in ("bf16", "f32"):
        for epilogue in (0, 1, 2):
            add(f"linear_{M}_{N}_{K}_{x}_{epilogue}", Linear(M, N, K, group, x, "f32" if M %% 2 else "bf16", epilogue, seed=M).run())
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
    assert normal.keys() == checked.keys() and len(normal) > 80
    for k in normal:
        assert normal[k] == checked[k], k
