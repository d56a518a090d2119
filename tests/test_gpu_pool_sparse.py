"""Attention over maps of which almost nothing is live, so that one list of 128 tokens spans a session (GB300)."""
import pytest
import torch

import pool_reference as ref
from test_gpu_pool import BF, I32, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import kv_cache_retention_gb300 as kv
    c = kv.Context(0)
    yield c
    c.check_device()
    c.close()


@pytest.mark.parametrize("new", [2, 100])  # few tokens; chunks
@pytest.mark.parametrize("n,Hkv", [(5000, 2), (1 << 20, 160)])
def test_nan_values_among_the_new_tokens_of_a_sparse_map(ctx, new, n, Hkv):
    """Several long sessions of some twenty live tokens and the new ones: NaN and infinite values among those reach the rows that
    see them, and the time that takes does not let the block's other waits run out (with so many kv heads a block has whole
    sessions, one after the other)."""
    S, D, page, old = 3, 64, 16, 20
    g = torch.Generator(device="cuda").manual_seed(n + new)
    P = S * (old + new) // page + 2
    k, v = (torch.randn((P, page, Hkv, D), generator=g, device="cuda").to(BF) for _ in range(2))
    q = torch.randn((S * new, 2 * Hkv, D), generator=g, device="cuda").to(BF)
    at = torch.cat([torch.arange(old, device="cuda") * ((n - new) // old), torch.arange(n - new, n, device="cuda")])
    free = torch.randperm(P * page, generator=g, device="cuda")[:S * (old + new)].view(S, -1)
    maps = torch.full((S, n), P * page, dtype=I32, device="cuda")
    maps[:, at] = free.to(I32)
    live = torch.zeros((S, n), dtype=torch.bool, device="cuda")
    live[:, at] = True
    cu, lens = [s * new for s in range(S + 1)], [n] * S

    def run(v):
        out, lse = torch.full_like(q, 9), torch.full(q.shape[:2], 9.0, device="cuda")
        ctx.pool_attention(q, k, v, _i32(cu), _i32(lens), out, slot_map=maps, dead_slot=P * page, lse=lse)
        ctx.check_device()
        return out, lse
    out, lse = run(v)
    ref.check_attend(out, lse, ref.attend(q, k, v, cu, lens, maps.long(), live, D ** -0.5))
    i, j = new // 2, new - 1
    bad = v.clone().flatten(0, 1)
    bad[free[:, old + i], 1, 7] = float("inf")
    bad[free[:, old + j], 1, 7] = -float("inf")
    bad[free[:, old + j], Hkv - 1, 60] = float("nan")
    got, got_lse = run(bad.view_as(v))
    assert torch.equal(got_lse, lse)
    rows, clean = got.view(S, new, 2 * Hkv, D), out.view(S, new, 2 * Hkv, D)
    if i < j:
        assert (rows[:, i:j, 2:4, 7] == float("inf")).all()
        assert torch.isnan(rows[:, j, 2:4, 7].float()).all()
    else:
        assert torch.isinf(rows[:, j, 2:4, 7].float()).all()
    assert torch.isnan(rows[:, j, -2:, 60].float()).all()
    same = torch.ones_like(rows, dtype=torch.bool)
    same[:, i:, 2:4, 7] = False
    same[:, j:, -2:, 60] = False
    assert torch.equal(rows[same], clean[same])
