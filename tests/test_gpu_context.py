"""A context made while the default stream is busy, and used at once on a stream that does not wait for that one."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import kv_cache_retention_gb300 as kv  # noqa: E402

I32, BF = torch.int32, torch.bfloat16


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _busy(ms):
    """About `ms` of work queued on the default stream (a kernel that counts clock cycles)."""
    torch.cuda._sleep(int(ms * 2e6))


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=I32).cuda()


def test_an_error_set_on_a_side_stream_is_not_cleared_later():
    x, out = torch.ones((8, 1, 64), dtype=BF, device="cuda"), torch.zeros((8, 1, 64), dtype=BF, device="cuda")
    bad, good = _i32([0, 9]), _i32([0, 8])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _busy(100)
    ctx = kv.Context(0)
    with torch.cuda.stream(side):
        ctx.prompt_attention(x, x, x, bad, out)
    side.synchronize()
    torch.cuda.synchronize()  # what the default stream held has run by now
    with pytest.raises(kv.KvselError, match="length out of range"):
        ctx.check_device()
    # the same after the word has been read and cleared
    with torch.cuda.stream(side):
        ctx.prompt_attention(x, x, x, bad, out)
        with pytest.raises(kv.KvselError, match="length out of range"):
            ctx.check_device()
        ctx.prompt_attention(x, x, x, bad, out)
    side.synchronize()
    torch.cuda.synchronize()
    with pytest.raises(kv.KvselError, match="length out of range"):
        ctx.check_device()
    ctx.prompt_attention(x, x, x, good, out)
    ctx.check_device()
    ctx.close()


def test_partial_results_of_a_new_context():
    """Sessions that several blocks share, attended on a side stream right after the context is made."""
    g = torch.Generator(device="cuda").manual_seed(1)
    S, Hq, Hkv, D, page, rows = 2, 8, 2, 128, 16, 256
    P = S * rows
    codes = lambda n: torch.randint(0, 256, (P, Hkv, page, n), generator=g, device="cuda").to(torch.uint8)  # noqa: E731
    scales = lambda n: torch.randint(100, 124, (P, Hkv, page, n), generator=g, device="cuda").to(torch.uint8)  # noqa: E731
    cache = [codes(D // 2), scales(D // 16), codes(D // 2), scales(D // 16)]
    table = torch.randperm(P, generator=g, device="cuda").to(I32).view(S, rows).contiguous()
    q = torch.randn((S, 1, Hq, D), generator=g, device="cuda").to(BF)
    lens = _i32([4000, 2111])
    ctx = kv.Context(0)
    want = torch.empty_like(q)
    ctx.kv4_attention(q, *cache, lens, want, block_table=table)
    ctx.check_device()
    ctx.close()
    side = torch.cuda.Stream()
    outs = [torch.empty_like(q) for _ in range(200)]
    torch.cuda.synchronize()
    _busy(2)  # ends while the calls below run
    ctx = kv.Context(0)
    with torch.cuda.stream(side):
        for o in outs:
            ctx.kv4_attention(q, *cache, lens, o, block_table=table)
    torch.cuda.synchronize()
    ctx.check_device()
    assert all(torch.equal(o, want) for o in outs)
    ctx.close()
