"""Attention and its weight per token in tables that reach almost 2^31 positions (GB300)."""
import pytest
import torch

import pool_reference as ref
from test_gpu_pool import BF, F32, I32, _i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import kv_cache_retention_gb300 as kv
    c = kv.Context(0)
    yield c
    c.check_device()
    c.close()


def test_mass_of_a_table_that_reaches_almost_2_31_positions(ctx):
    """The score's rows are written to their ends and not outside: the copy's step past the last position passes 2^31."""
    page, rows, n, new, D = 1 << 17, (1 << 14) - 1, 300, 3, 64
    reach = page * rows
    assert 2 ** 31 - 2 ** 18 < reach < 2 ** 31 - 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((1, page, 1, D), generator=g, device="cuda").to(BF) for _ in range(2))
    q = torch.randn((new, 2, D), generator=g, device="cuda").to(BF)
    table = torch.full((1, rows), -1, dtype=I32, device="cuda")
    table[0, 0] = 0
    cu, lens, out, lse = _i32([0, new]), _i32([n]), torch.empty_like(q), torch.empty((new, 2), device="cuda")
    ctx.pool_attention(q, k, v, cu, lens, out, block_table=table, lse=lse)
    slots, live = torch.arange(n, device="cuda")[None], torch.ones((1, n), dtype=torch.bool, device="cuda")
    ref.check_attend(out, lse, ref.attend(q, k, v, [0, new], [n], slots, live, D ** -0.5))
    # rows of the score between two stretches that nothing may write
    held = torch.full((reach + 2 * 1024,), 7.0, dtype=F32, device="cuda")
    score, before = held[1024:1024 + reach].view(1, reach), torch.full((1, reach), 3.0, device="cuda")
    for given, base in ((before, 3.0), (None, 0.0)):
        ctx.attention_mass(q, lse, k, cu, lens, score, block_table=table, score_in=given)
        ctx.check_device()
        want = ref.mass(q, lse, k, [0, new], [n], slots, live, D ** -0.5, torch.full((1, n), base, device="cuda"))
        ref.check_mass(score[:, :n], want)
        assert (held[:1024] == 7).all() and (held[1024 + reach:] == 7).all()
        low, high = torch.aminmax(score[:, n:])
        assert float(low) == float(high) == base
