"""A process whose first calls over the page pools are captured into a graph, with no call before them."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

PROGRAM = r"""
import sys
import torch
sys.path.insert(0, "tests")
import numpy as np
import kv_cache_retention_gb300 as kv
import pool_reference as ref
from test_gpu_pool import World, _i32

ctx = kv.Context(0)
worlds = [World(new, lens, Hq, Hkv, D, 16, kind, seed=3) for new, lens, Hq, Hkv, D, kind in (
    ([1, 1], [2000, 900], 8, 2, 128, "map"), ([1, 2], [700, 33], 6, 3, 64, "table"),
    ([300, 40], [1500, 40], 8, 2, 64, "map"), ([200], [1000], 4, 1, 128, "table"))]
scores = [torch.empty((w.S, w.slots.shape[1]), device="cuda") for w in worlds]
w0 = worlds[0]
budget, out_map = _i32([500, 2000]), torch.empty_like(w0.args["slot_map"])
before = w0.args["slot_map"].cpu().numpy()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for w, s in zip(worlds, scores):
        w.attend(ctx)
        ctx.attention_mass(w.q, w.lse, w.k, w.cu, w.lens, s, scale=w.scale, **w.args)
    ctx.evict_slots(scores[0], w0.lens, budget, w0.args["slot_map"], w0.dead, out_map)
first = None
for _ in range(2):
    for t in [x for w, s in zip(worlds, scores) for x in (w.out, w.lse, s)] + [out_map]:
        t.fill_(9)
    graph.replay()
    ctx.check_device()
    got = [x.clone() for w, s in zip(worlds, scores) for x in (w.out, w.lse, s)] + [out_map.clone()]
    assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
    first = got
    for w, s in zip(worlds, scores):
        ref.check_attend(w.out, w.lse, w.want())
        ref.check_mass(s, ref.mass(w.q, w.lse, w.k, w.cu_host, w.lens_host, w.slots, w.live, w.scale, torch.zeros_like(s)))
    want, _, _ = ref.evict(scores[0].cpu().numpy(), w0.lens.tolist(), budget.tolist(), before, w0.dead, 0, 0)
    assert np.array_equal(out_map.cpu().numpy(), want)
ctx.close()
print("captured first")
"""


def test_first_pool_calls_are_captured():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-3000:]
