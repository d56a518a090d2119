"""Decode steps of sessions whose slot maps were pruned: steps planned without maps leave what redirect_slots dropped
dropped, their new slots go to the maps' rows."""
import numpy as np
import pytest
import torch

from test_gpu_serving import _attention_reference, _check_attention, _i32, _random_cache

pytestmark = pytest.mark.gpu

import kv_cache_retention_gb300 as kv  # noqa: E402

I32, BF = torch.int32, torch.bfloat16


def test_pruned_maps_stay_over_planned_steps():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ctx = kv.Context(0)
    g = torch.Generator(device="cuda").manual_seed(7)
    page, Hq, Hkv, D, S, rows, P, dead = 16, 8, 2, 64, 3, 10, 40, 40 * 16
    cache = _random_cache(g, P, Hkv, page, D)
    lens = [70, 33, 128]
    table = torch.full((S, rows), -1, dtype=I32, device="cuda")
    maps = torch.empty((S, rows * page), dtype=I32, device="cuda")
    free = torch.randperm(P, generator=g, device="cuda").to(I32)
    counts = torch.empty(2, dtype=I32, device="cuda")
    cu, slots, pos = (torch.empty(n, dtype=I32, device="cuda") for n in (S + 1, sum(lens), sum(lens)))
    ctx.plan_slots(_i32([0] * S), _i32(lens), free, page, P, table, cu, slots, pos, counts, slot_map=maps)
    full = maps.cpu().numpy()
    rng = np.random.default_rng(7)
    kept = np.ones((S, rows * page), bool)
    for s in (0, 2):
        kept[s, :lens[s]] = rng.random(lens[s]) < 0.3
        ctx.redirect_slots(maps[s, :lens[s]], torch.from_numpy(kept[s, :lens[s]].astype(np.uint8)).cuda(), dead,
                           maps[s, :lens[s]])
    sessions = torch.arange(S, device="cuda")
    for _ in range(3):
        free = free[int(counts[1]):].contiguous()
        cu, slots, pos = (torch.empty(n, dtype=I32, device="cuda") for n in (S + 1, S, S))
        ctx.plan_slots(_i32(lens), _i32([1] * S), free, page, P, table, cu, slots, pos, counts)
        maps[sessions, pos.long()] = slots
        for s in range(S):
            full[s, lens[s]] = int(slots[s])
        lens = [n + 1 for n in lens]
        x = torch.randn((S, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
        ctx.kv4_store(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots, *cache)
        q = x[:, :Hq].unsqueeze(1)
        out, lse = torch.empty((S, 1, Hq, D), dtype=BF, device="cuda"), torch.empty((S, 1, Hq), device="cuda")
        ctx.kv4_attention(q, *cache, _i32(lens), out, slot_map=maps, dead_slot=dead, lse=lse)
        ctx.check_device()
        assert np.array_equal(maps.cpu().numpy(), np.where(kept, full, dead))
        _check_attention(out, lse, _attention_reference(q, cache, lens, np.where(full < 0, 0, full), kept & (full >= 0),
                                                        D ** -0.5))
    ctx.close()


def test_tokens_that_do_not_fit():
    """What is cut and what is not: a table row cuts a length everywhere; new_slots and a map's row leave tokens out."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ctx = kv.Context(0)

    def plan(cached, new, max_blocks, T, ld):
        table = torch.full((len(new), max_blocks), -1, dtype=I32, device="cuda")
        cu, slots, pos, counts = (torch.full((n,), -7, dtype=I32, device="cuda") for n in (len(new) + 1, T, T, 2))
        maps = torch.full((len(new), ld), -7, dtype=I32, device="cuda")
        ctx.plan_slots(_i32(cached), _i32(new), _i32(range(8)), 4, 8, table, cu, slots, pos, counts, slot_map=maps)
        with pytest.raises(kv.KvselError, match="length out of range"):
            ctx.check_device()
        return table.tolist(), cu.tolist(), slots.tolist(), pos.tolist(), counts.tolist(), maps.tolist()

    # 9 tokens in a table row of two pages of four: cut to 8 in every output
    assert plan([0], [9], 2, 10, 8) == ([[0, 1]], [0, 8], [*range(8), -1, -1], [*range(8), -1, -1], [8, 2], [[*range(8)]])
    # 9 tokens, new_slots of 5, and then a map's row of 6: the rest is left out, the lengths stay
    assert plan([0], [9], 3, 5, 9) == ([[0, 1, 2]], [0, 9], [*range(5)], [*range(5)], [9, 3], [[*range(9)]])
    assert plan([0], [9], 3, 9, 6) == ([[0, 1, 2]], [0, 9], [*range(9)], [*range(9)], [9, 3], [[*range(6)]])
    ctx.close()
