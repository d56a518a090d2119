"""Attention over the 4-bit cache where a block takes several pieces of sessions one after the other, and where a piece's
tokens come to shared memory in both ways, as runs and one by one."""
import numpy as np
import pytest
import torch

from test_gpu_serving import _attention_reference, _check_attention, _i32, _random_cache

pytestmark = pytest.mark.gpu

import kv_cache_retention_gb300 as kv  # noqa: E402

I32, BF = torch.int32, torch.bfloat16


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    c = kv.Context(0)
    yield c
    c.check_device()
    c.close()


def _repeated(ctx, q, cache, lens, times, **args):
    """The call's outputs, which are the same each time."""
    S, Tq, Hq, _ = q.shape
    first = None
    for _ in range(times):
        out, lse = torch.full_like(q, 9), torch.full((S, Tq, Hq), 9.0, device="cuda")
        ctx.kv4_attention(q, *cache, lens, out, lse=lse, **args)
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    ctx.check_device()
    return first


@pytest.mark.parametrize("D,Tq,Hq,Hkv", [(64, 1, 16, 8), (128, 1, 16, 8), (128, 4, 16, 8), (256, 1, 8, 8)])
@pytest.mark.parametrize("reach", [640, 1600])
def test_runs_and_single_tokens_in_turn(ctx, D, Tq, Hq, Hkv, reach):
    """Slot maps whose runs of 32 slots alternate with scattered ones, in more sessions than blocks hold at a time."""
    g = torch.Generator(device="cuda").manual_seed(D + reach)
    rng = np.random.default_rng(D + reach)
    S, page, P = 90, 16, 200
    cache = _random_cache(g, P, Hkv, page, D)
    q = torch.randn((S, Tq, Hq, D), generator=g, device="cuda").to(BF)
    slots = np.empty((S, reach), np.int64)
    for s in range(S):
        for c in range(0, reach, 32):
            run = (c // 32 + s) % 3
            start = int(rng.integers(0, P * page // 16 - 2)) * 16
            slots[s, c:c + 32] = start + np.arange(32) if run else rng.integers(0, P * page, 32)
    live = np.ones_like(slots, bool)
    lens = [int(n) for n in rng.integers(1, reach + 1, S)]
    lens[3], lens[17] = 0, reach
    out, lse = _repeated(ctx, q, cache, _i32(lens), 25, slot_map=_i32(slots))
    rows = sorted(rng.choice(S, 12, replace=False).tolist() + [3, 17])
    _check_attention(out[rows], lse[rows], _attention_reference(q[rows], cache, [lens[s] for s in rows], slots[rows],
                                                                live[rows], D ** -0.5))
