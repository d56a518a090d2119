"""The lists of live tokens that the calls over the page pools go by: their last, partly filled groups (GB300)."""
import pytest
import torch

from test_gpu_pool import I32, World

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import kv_cache_retention_gb300 as kv
    c = kv.Context(0)
    yield c
    c.check_device()
    c.close()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 20, 100])  # few tokens; a chunk of one tile; of two
@pytest.mark.parametrize("tokens", [31, 47, 127])
def test_values_behind_a_list_that_ends_in_a_run(ctx, D, new, tokens):
    """A list whose last 15 tokens lie on consecutive slots, the next of which is its first token's: that token's row, infinite
    in one value, counts once and not again as a row behind the list's end (0 * inf)."""
    n = tokens + new                    # the new tokens themselves are dropped: every row sees the whole list
    w = World([new], [n], 8, 2, D, 16, "table", seed=tokens)
    free = torch.randperm(w.P * 16, device="cuda")
    first = 48
    free = free[(free < first) | (free >= first + 16)]
    slots = torch.full((1, n), -1, dtype=torch.int64, device="cuda")
    slots[0, :tokens] = free[:tokens]
    slots[0, tokens - 15:tokens] = torch.arange(first, first + 15, device="cuda")
    slots[0, 0] = first + 15
    w.v.flatten(0, 1)[first + 15, 0, 3] = float("inf")
    w.attend(ctx, block_table=None, slot_map=slots.to(I32))
    ctx.check_device()
    got = w.out.float()
    assert (got[:, :4, 3] == float("inf")).all()
    got[:, :4, 3] = 0
    assert torch.isfinite(got).all()
