"""Bounded waits of the serving kernels that run out, made to do so without faulting or hanging the GPU: internal entries
let one warp of every block wait, with a limit of 2 ms, on a barrier that nothing completes, while the block's own copies
are on their way.  The call reports the timeout, and the next calls on the same context are right."""
import ctypes

import pytest
import torch

from test_gpu_serving import _i32, _random_cache

pytestmark = pytest.mark.gpu

import kv_cache_retention_gb300 as kv  # noqa: E402

I32, BF = torch.int32, torch.bfloat16
LIMIT = 2_000_000


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    c = kv.Context(0)
    yield c
    c.check_device()
    c.close()


def _entry(name, like):
    """The test entry `name`: the arguments of the public call `like` with the limit before the stream."""
    fn = getattr(kv._lib, name)
    fn.restype, args = kv.SIGNATURES[like]
    fn.argtypes = [*args[:-1], ctypes.c_uint64, args[-1]]
    return fn


@pytest.mark.parametrize("kind", ["table", "map"])
@pytest.mark.parametrize("S,Tq,Hq,Hkv,D,n", [(2, 1, 8, 2, 128, 4000), (3, 4, 16, 4, 128, 2500), (5, 1, 4, 2, 64, 600), (2, 1, 4, 2, 256, 1500)])
def test_kv4_attention_gives_up_and_recovers(ctx, S, Tq, Hq, Hkv, D, n, kind):
    give_up = _entry("kvsel_test_kv4_attention_give_up", "kvsel_kv4_attention")
    g = torch.Generator(device="cuda").manual_seed(n)
    rows = n // 16 + 1
    cache = _random_cache(g, S * rows, Hkv, 16, D)
    q = torch.randn((S, Tq, Hq, D), generator=g, device="cuda").to(BF)
    lens = _i32([n - 100 * s for s in range(S)])
    table = torch.randperm(S * rows, generator=g, device="cuda").to(I32).view(S, rows).contiguous()
    tokens = table
    if kind == "map":
        tokens = (table[:, :, None] * 16 + torch.arange(16, dtype=I32, device="cuda")).view(S, rows * 16).contiguous()
    want, out = torch.empty_like(q), torch.empty_like(q)
    args = dict(block_table=tokens) if kind == "table" else dict(slot_map=tokens)
    ctx.kv4_attention(q, *cache, lens, want, **args)
    ctx.check_device()
    s = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        rc = give_up(ctx.handle, q.data_ptr(), Hq * D, S, Tq, Hq, Hkv, D, *[c.data_ptr() for c in cache], S * rows, 16,
                     lens.data_ptr(), tokens.data_ptr() if kind == "map" else None,
                     tokens.data_ptr() if kind == "table" else None, tokens.shape[1], -1, D ** -0.5, out.data_ptr(), None,
                     LIMIT, s)
        assert rc == kv.OK, kv.kvsel_last_error_string(ctx.handle)
        assert kv.kvsel_check_device(ctx.handle, s) == kv.ERR_TIMEOUT, kv.kvsel_last_error_string(ctx.handle)
        ctx.kv4_attention(q, *cache, lens, out, **args)
        ctx.check_device()
        assert torch.equal(out, want)


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([600, 90, 1, 300], 8, 2, 128), ([500] * 12, 32, 8, 64), ([300, 40], 2, 2, 64)])
def test_prompt_attention_gives_up_and_recovers(ctx, lens, Hq, Hkv, D):
    give_up = _entry("kvsel_test_prompt_attention_give_up", "kvsel_prompt_attention")
    g = torch.Generator(device="cuda").manual_seed(len(lens))
    T = sum(lens)
    q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    cu = _i32([sum(lens[:i]) for i in range(len(lens) + 1)])
    want, out = torch.empty_like(q), torch.empty_like(q)
    ctx.prompt_attention(q, k, v, cu, want)
    ctx.check_device()
    s = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        rc = give_up(ctx.handle, q.data_ptr(), k.data_ptr(), v.data_ptr(), Hq * D, Hkv * D, Hkv * D, cu.data_ptr(), len(lens),
                     T, Hq, Hkv, D, D ** -0.5, out.data_ptr(), None, LIMIT, s)
        assert rc == kv.OK, kv.kvsel_last_error_string(ctx.handle)
        assert kv.kvsel_check_device(ctx.handle, s) == kv.ERR_TIMEOUT, kv.kvsel_last_error_string(ctx.handle)
        ctx.prompt_attention(q, k, v, cu, out)  # tensor memory is free again
        ctx.check_device()
        assert torch.equal(out, want)


def test_give_up_entries_reject_bad_limits(ctx):
    give_up = _entry("kvsel_test_kv4_attention_give_up", "kvsel_kv4_attention")
    s = torch.cuda.current_stream().cuda_stream
    for wait in (0, 2_000_000_000):
        assert give_up(ctx.handle, None, 128, 1, 1, 1, 1, 128, None, None, None, None, 1, 16, None, None, None, 1, -1, 1.0,
                       None, None, wait, s) == kv.ERR_INVALID_ARG
    give_up = _entry("kvsel_test_prompt_attention_give_up", "kvsel_prompt_attention")
    for wait in (0, 2_000_000_000):
        assert give_up(ctx.handle, None, None, None, 128, 128, 128, None, 1, 1, 1, 1, 128, 1.0, None, None, wait,
                       s) == kv.ERR_INVALID_ARG
