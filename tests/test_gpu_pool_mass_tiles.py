"""attention_mass where an ordinary product does not fill its tile: groups whose heads leave rows of a tile of 128 over, and the
columns of tensor memory that no product has written (GB300)."""
import pytest
import torch

import pool_reference as ref
from test_gpu_pool import F32, World

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import kv_cache_retention_gb300 as kv
    c = kv.Context(0)
    yield c
    c.check_device()
    c.close()


def _lse(w):
    return torch.nan_to_num(w.want()[1], nan=0.0, neginf=-float("inf")).to(F32)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [64, 65, 71, 100, 112, 113, 128])
@pytest.mark.parametrize("n", [700, 60000])
def test_one_token_of_a_large_group(ctx, G, D, n):
    """One new token of up to 128 heads on one kv head: its product has as many columns as heads, and what the attention
    before it has left in tensor memory beside them (infinite weights of rows of no token) has no part in the sums."""
    w = World([1], [n], G, 1, D, 16, "table", seed=G)
    lse, score = _lse(w), torch.empty((1, w.slots.shape[1]), device="cuda")
    for _ in range(3):
        w.attend(ctx)
        ctx.attention_mass(w.q, lse, w.k, w.cu, w.lens, score, scale=w.scale, **w.args)
        ctx.check_device()
        ref.check_mass(score, ref.mass(w.q, lse, w.k, w.cu_host, w.lens_host, w.slots, w.live, w.scale, torch.zeros_like(score)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 3, 4, 5, 7, 10, 22, 40, 43, 65, 100])
@pytest.mark.parametrize("new", [1, 150])
def test_minus_infinite_logits(ctx, G, D, new):
    """Keys with an infinite element whose logits are -inf for every row have no weight, whatever the group's size leaves of
    a tile: their scores stay, and the others' are what they are without them."""
    n = 900
    w = World([new], [n], 2 * G, 2, D, 16, "table", seed=G)
    w.q[..., 0] = 1
    hidden = w.slots[0, 200:450]
    w.k.flatten(0, 1)[hidden] = 0
    w.k.flatten(0, 1)[hidden, :, 0] = -float("inf")
    live = torch.ones_like(w.live)
    live[0, 200:450] = False
    clean = w.k.clone()
    clean.flatten(0, 1)[hidden] = 0
    lse = ref.attend(w.q, clean, w.v, w.cu_host, w.lens_host, w.slots, live, w.scale)[1].to(F32)
    before = torch.rand((1, w.slots.shape[1]), device="cuda")
    score = torch.empty_like(before)
    ctx.attention_mass(w.q, lse, w.k, w.cu, w.lens, score, score_in=before, scale=w.scale, **w.args)
    ctx.check_device()
    assert torch.equal(score[0, 200:450], before[0, 200:450])
    ref.check_mass(score, ref.mass(w.q, lse, clean, w.cu_host, w.lens_host, w.slots, live, w.scale, before))
