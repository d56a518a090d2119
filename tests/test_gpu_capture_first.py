"""A process whose first serving calls are captured into a graph, with no call before them."""
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
import kv_cache_retention_gb300 as kv
from test_gpu_serving import _attention_reference, _check_attention, _check_prompt, _i32
import numpy as np

I32, BF = torch.int32, torch.bfloat16
ctx = kv.Context(0)
S, page, rows, Hq, Hkv, D = 2, 16, 100, 8, 2, 128
T = 1500
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
new, cached = _i32([1300, 200]), _i32([0, 0])
free = torch.randperm(S * rows, generator=g, device="cuda").to(I32)
table = torch.full((S, rows), -1, dtype=I32, device="cuda")
maps = torch.empty((S, rows * page), dtype=I32, device="cuda")
cu, slots, pos, counts = (torch.empty(n, dtype=I32, device="cuda") for n in (S + 1, T, T, 2))
cache = [torch.zeros((S * rows, Hkv, page, n), dtype=torch.uint8, device="cuda") for n in (64, 8, 64, 8)]
out, lse = torch.empty((T, Hq, D), dtype=BF, device="cuda"), torch.empty((T, Hq), device="cuda")
kb, vb = (torch.empty((T, Hkv, D), dtype=BF, device="cuda") for _ in range(2))
q1 = torch.randn((S, 1, Hq, D), generator=g, device="cuda").to(BF)
o1, o2 = torch.empty_like(q1), torch.empty_like(q1)
l1, l2 = (torch.empty((S, 1, Hq), device="cuda") for _ in range(2))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    ctx.plan_slots(cached, new, free, page, S * rows, table, cu, slots, pos, counts, slot_map=maps)
    ctx.prompt_attention(q, k, v, cu, out, lse=lse)
    ctx.kv4_store(k, v, slots, *cache)
    ctx.kv4_load(*cache, slots, kb, vb)
    ctx.kv4_attention(q1, *cache, new, o1, block_table=table, lse=l1)
    ctx.kv4_attention(q1, *cache, new, o2, slot_map=maps, lse=l2)
for _ in range(2):
    for t in (out, o1, o2):
        t.fill_(9)
    graph.replay()
    ctx.check_device()
    _check_prompt(q, k, v, [0, 1300, 1500], D ** -0.5, out, lse, rows=[0, 127, 128, 700, 1299, 1300, 1499])
    m = maps.cpu().numpy()
    want = _attention_reference(q1, cache, [1300, 200], np.where(m < 0, 0, m), m >= 0, D ** -0.5)
    _check_attention(o1, l1, want)
    _check_attention(o2, l2, want)
ctx.close()
print("captured first")
"""


def test_first_calls_are_captured():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-3000:]
