"""The 64-bit reference of the calls over the page pools against loops over single values, the refusal of a null context, and
the cutting of the sessions' lists into shares: every list in exactly one share, every joined unit's sharers counted (CPU)."""
import math
import random

import numpy as np
import torch

import pool_reference as ref


def _small(seed=0):
    g = torch.Generator().manual_seed(seed)
    new, lens, Hq, Hkv, D, page = [3, 0, 2], [7, 4, 1], 4, 2, 64, 4
    cu = [0, 3, 3, 5]
    q = torch.randn((6, Hq, D), generator=g).to(torch.bfloat16)
    k, v = (torch.randn((5, page, Hkv, D), generator=g).to(torch.bfloat16) for _ in range(2))
    slots = torch.randperm(20, generator=g)[:18].view(3, 6).repeat(1, 2)[:, :8].contiguous()
    live = torch.rand((3, 8), generator=g) < 0.7
    live[0, 2] = True
    return q, k, v, cu, lens, slots, live, new, Hq, Hkv, D, page


def test_reference_against_loops():
    q, k, v, cu, lens, slots, live, new, Hq, Hkv, D, page = _small()
    out, lse, _, _ = ref.attend(q, k, v, cu, lens, slots, live, 0.2)
    before = torch.rand((3, 8))
    score, _ = ref.mass(q, torch.nan_to_num(lse, nan=0.0, neginf=-math.inf), k, cu, lens, slots, live, 0.2, before)
    want = before.double().clone()
    for s in range(3):
        for i in range(new[s]):
            pos = lens[s] - new[s] + i
            for h in range(Hq):
                seen = [j for j in range(lens[s]) if live[s, j] and j <= pos]
                row = q[cu[s] + i, h].double()
                x = [0.2 * float(row @ k[slots[s, j] // page, slots[s, j] % page, h // 2].double()) for j in seen]
                total = math.log(sum(math.exp(y) for y in x)) if x else -math.inf
                assert (math.isinf(total) and torch.isinf(lse[cu[s] + i, h])) or abs(float(lse[cu[s] + i, h]) - total) < 1e-12
                o = sum((math.exp(y - total) * v[slots[s, j] // page, slots[s, j] % page, h // 2].double() for y, j in zip(x, seen)),
                        torch.zeros(D, dtype=torch.float64))
                assert torch.allclose(out[cu[s] + i, h], o, rtol=0, atol=1e-12)
                for y, j in zip(x, seen):
                    want[s, j] += math.exp(y - total)
    assert torch.isnan(out[5]).all() and torch.allclose(score, want, rtol=0, atol=1e-12)


def test_evict_by_hand():
    score = np.array([[5, 1, 1, 9, 0, 1, np.nan, 2]], np.float32)
    slots = [[10, 11, 12, 13, 14, 15, 16, 17]]
    # a NaN leaves first, then 0, then the last of the ones; positions 0 and 7 are protected
    out, freed, n = ref.evict(score, [8], [5], slots, 99, 1, 1)
    assert freed == [[14, 15, 16]] and n == [3] and out.tolist() == [[10, 11, 12, 13, 99, 99, 99, 17]]
    out, freed, n = ref.evict(score, [8], [5], slots, 99, 1, 1, room=2)
    assert freed == [[14, 16]] and n == [2]
    assert ref.evict(score, [8], [0], slots, 99, 4, 4)[2] == [0]


def test_null_context():
    import kv_cache_retention_gb300 as kv
    assert kv.kvsel_pool_attention(None, None, 128, None, 1, 1, 1, 1, 128, None, None, 128, 128, 1, 16, None, None, None, 1, -1, 1.0,
                                   None, None, None) == kv.ERR_INVALID_ARG
    assert kv.kvsel_attention_mass(None, None, 128, None, None, 1, 1, 1, 1, 128, None, 128, 1, 16, None, None, None, 1, -1, 1.0, None,
                                   None, 16, None) == kv.ERR_INVALID_ARG
    assert kv.kvsel_evict_slots(None, None, 8, None, None, 1, None, 8, 9, 0, 0, None, None, 0, None, None) == kv.ERR_INVALID_ARG


TILE = 128


def _pieces(units, shares, start, least):
    """The kernels' cutting: units [(size of its work, lists)], laid end to end -> pieces (share, unit, first list, stop), and
    for each unit that a share starts without ending it, the sharers that the share counts."""
    total = sum(size for size, _ in units)
    quota = max(-(-total // shares), least * TILE)
    pieces, joints = [], {}
    for share in range(shares):
        lo, hi, at = share * quota, (share + 1) * quota, 0
        for k, (size, lists) in enumerate(units):
            u0, u1 = at, at + size
            at = u1
            if size == 0 or u1 <= lo or u0 >= hi:
                continue
            list_at = lambda p: min(lists, max(0, (p - u0) // TILE - start))  # noqa: E731
            l0 = 0 if lo <= u0 else list_at(lo)
            l1 = lists if hi >= u1 else list_at(hi)
            if l0 >= l1:
                continue
            pieces.append((share, k, l0, l1))
            if l0 == 0 and l1 < lists:
                assert share not in joints
                joints[share] = (k, (min(u1, u0 + (lists + start) * TILE) - 1) // quota - share + 1)
    return pieces, joints


def test_shares_cover_every_list_once():
    rng = random.Random(3)
    for trial in range(400):
        shares, start, least = rng.choice([1, 2, 9, 19, 38, 152]), rng.choice([2, 4]), rng.choice([1, 4])
        units = []
        for _ in range(rng.randint(1, 40)):
            few = rng.random() < 0.5
            length = rng.choice([0, 1, 127, 128, 129, rng.randint(0, 3000), rng.randint(0, 40000)])
            if few:                                   # a session of few tokens
                units.append((length + start * TILE, max(1, -(-length // TILE))))
            else:                                     # units of `unit` tokens, the last one counted as if it were full
                unit, count = rng.choice([2, 50, 64, 256]), rng.randint(0, 700)
                base = max(0, length - count)
                for t in range(-(-count // unit)):
                    keys = max(0, length - count + min(count, (t + 1) * unit))
                    units.append((base + start * TILE + (t + 1) * unit, max(1, -(-keys // TILE))))
        pieces, joints = _pieces(units, shares, start, least)
        for k, (size, lists) in enumerate(units):
            mine = [p for p in pieces if p[1] == k]
            if size == 0:
                assert not mine
                continue
            assert [p[2] for p in mine] == [0] + [p[3] for p in mine[:-1]] and mine[-1][3] == lists, (trial, k)
            assert [p[0] for p in mine] == list(range(mine[0][0], mine[0][0] + len(mine)))
            if len(mine) > 1:
                assert joints[mine[0][0]] == (k, len(mine))
            else:
                assert joints.get(mine[0][0], (None,))[0] != k
        # a share has one unit that began before it at most (its first) and one that goes on behind it (its last)
        for share in range(shares):
            own = [p for p in pieces if p[0] == share]
            assert all(p[2] == 0 for p in own[1:]) and all(p[3] == units[p[1]][1] for p in own[:-1])


def test_page_of_a_position_by_multiplication():
    """The quotient of a position by the page size, as the calls' tables use it: (2^(31+l) / page + 1) j >> (31 + l)."""
    rng = random.Random(4)
    for _ in range(20000):
        page = rng.choice([rng.randint(2, 300), rng.randint(2, 2 ** 31 - 1), 2 ** rng.randint(1, 30), 2 ** rng.randint(2, 30) + rng.choice([-1, 1])])
        bits = 1
        while (1 << bits) < page:
            bits += 1
        mul = (1 << (31 + bits)) // page + 1
        assert mul < 1 << 32
        near = rng.randint(0, (2 ** 31 - 1) // page) * page
        for j in (0, rng.randint(0, 2 ** 31 - 1), 2 ** 31 - 1, near, max(0, near - 1)):
            assert (j * mul) >> (31 + bits) == j // page
