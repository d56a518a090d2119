"""Attention over the 4-bit cache where a block takes several pieces of sessions one after the other, and where a piece's
tokens come to shared memory in both ways, as runs and one by one."""
import numpy as np
import pytest
import torch

from test_gpu_serving import _attention_reference, _check_attention, _i32, _random_cache
from test_gpu_serving import test_attention_matches_reference as _matches_reference

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
        assert torch.equal(out.view(torch.int16), first[0].view(torch.int16))  # by their bits: a NaN equals itself
        assert torch.equal(lse.view(I32), first[1].view(I32))
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


SHARED = [
    # S, Tq, Hq, Hkv, D, page, lens: units that several blocks share, joined from partial results
    (3, 4, 16, 4, 128, 16, [2500, 301, 1700]),      # two row tiles, blocks of six warps
    (1, 2, 16, 2, 128, 16, [9000]),
    (2, 12, 12, 2, 128, 16, [1900, 1100]),          # several tiles of 16 rows, the last one not full
    (2, 1, 8, 2, 256, 16, [1500, 900]),
    (2, 1, 12, 1, 256, 16, [1500, 1201]),           # more rows than a tile
    (3, 3, 4, 2, 256, 7, [2600, 1, 1400]),
    (2, 4, 12, 2, 64, 16, [2000, 1100]),
    (1, 5, 16, 1, 64, 48, [5000]),
    (1, 1, 1, 1, 256, 16, [6000]),
    (2, 320, 16, 16, 64, 16, [1100, 900]),          # more units than blocks: one share, units in turn
    (1, 256, 19, 19, 64, 16, [900]),
    (2, 160, 8, 8, 256, 16, [1030, 200]),
    (1, 310, 16, 16, 128, 16, [900]),
]


@pytest.mark.parametrize("S,Tq,Hq,Hkv,D,page,lens", SHARED)
@pytest.mark.parametrize("kind", ["table", "map"])
def test_shared_units_match_reference(ctx, S, Tq, Hq, Hkv, D, page, lens, kind):
    _matches_reference(ctx, S, Tq, Hq, Hkv, D, page, lens, kind)
    assert -(-max(lens) // page) * page > 768  # what a row of the map or table reaches: units are not taken whole


@pytest.mark.parametrize("D,G", [(64, 2), (128, 4), (256, 1)])
def test_nan_in_the_last_tokens_of_shared_units(ctx, D, G):
    """Drafted rows: a NaN value group of a late token reaches the rows that see it and no others, through the join."""
    g = torch.Generator(device="cuda").manual_seed(D)
    S, Tq, Hkv, page, lens = 2, 6, 2, 16, [3000, 1300]
    rows = 200
    cache = _random_cache(g, S * rows, Hkv, page, D)
    q = torch.randn((S, Tq, Hkv * G, D), generator=g, device="cuda").to(BF)
    table = torch.randperm(S * rows, generator=g, device="cuda").to(I32).view(S, rows).contiguous()
    clean, _ = _repeated(ctx, q, cache, _i32(lens), 1, block_table=table)
    for s, back in ((0, 4), (1, 1)):                # the token `back` places before the session's end
        at = lens[s] - back
        cache[3][int(table[s, at // page]), 1, at % page, 2] = 255
    out, lse = _repeated(ctx, q, cache, _i32(lens), 5, block_table=table)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, Tq - 4:, G:, 32:48] = hit[1, Tq - 1:, G:, 32:48] = True
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit]) and torch.isfinite(lse).all()
