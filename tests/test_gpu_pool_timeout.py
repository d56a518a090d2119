"""Bounded waits of the calls over the page pools that run out, made to do so without faulting or hanging the GPU: internal
entries let one issuing warp of every block wait, with a limit of 2 ms, on a barrier that nothing completes, while the
block's own copies are on their way.  The call reports the timeout, and the next calls on the same context are right."""
import ctypes

import pytest
import torch

from test_gpu_pool import World

pytestmark = pytest.mark.gpu

LIMIT = 2_000_000


@pytest.fixture(scope="module")
def ctx():
    import kv_cache_retention_gb300 as kv
    c = kv.Context(0)
    yield c
    c.check_device()
    c.close()


def _entry(name, like):
    import kv_cache_retention_gb300 as kv
    fn = getattr(kv._lib, name)
    fn.restype, args = kv.SIGNATURES[like]
    fn.argtypes = [*args[:-1], ctypes.c_uint64, args[-1]]
    return fn


def _map_args(w):
    sm, bt = w.args.get("slot_map"), w.args.get("block_table")
    t = sm if sm is not None else bt
    return (None if sm is None else sm.data_ptr(), None if bt is None else bt.data_ptr(), t.shape[1], w.args.get("dead_slot", -1))


CASES = [([1, 1], [4000, 900], 8, 2, 128), ([300, 1, 40], [2500, 600, 50], 6, 2, 64), ([500], [5000], 32, 8, 128)]


@pytest.mark.parametrize("kind", ["table", "map"])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D", CASES)
def test_pool_attention_gives_up_and_recovers(ctx, new, lens, Hq, Hkv, D, kind):
    import kv_cache_retention_gb300 as kv
    give_up = _entry("kvsel_test_pool_attention_give_up", "kvsel_pool_attention")
    w = World(new, lens, Hq, Hkv, D, 16, kind, seed=40)
    w.attend(ctx)
    ctx.check_device()
    want = w.out.clone()
    s = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        rc = give_up(ctx.handle, w.q.data_ptr(), Hq * D, w.cu.data_ptr(), w.S, w.q.shape[0], Hq, Hkv, D, w.k.data_ptr(),
                     w.v.data_ptr(), Hkv * D, Hkv * D, w.P, 16, w.lens.data_ptr(), *_map_args(w), w.scale, w.out.data_ptr(), None,
                     LIMIT, s)
        assert rc == kv.OK, kv.kvsel_last_error_string(ctx.handle)
        assert kv.kvsel_check_device(ctx.handle, s) == kv.ERR_TIMEOUT, kv.kvsel_last_error_string(ctx.handle)
        w.attend(ctx)  # tensor memory is free again
        ctx.check_device()
        assert torch.equal(w.out, want)


@pytest.mark.parametrize("kind", ["table", "map"])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D", CASES)
def test_attention_mass_gives_up_and_recovers(ctx, new, lens, Hq, Hkv, D, kind):
    import kv_cache_retention_gb300 as kv
    give_up = _entry("kvsel_test_attention_mass_give_up", "kvsel_attention_mass")
    w = World(new, lens, Hq, Hkv, D, 16, kind, seed=41)
    w.attend(ctx)
    score = torch.empty((w.S, w.slots.shape[1]), device="cuda")
    call = lambda: ctx.attention_mass(w.q, w.lse, w.k, w.cu, w.lens, score, scale=w.scale, **w.args)  # noqa: E731
    call()
    ctx.check_device()
    want = score.clone()
    s = torch.cuda.current_stream().cuda_stream
    for _ in range(2):
        rc = give_up(ctx.handle, w.q.data_ptr(), Hq * D, w.lse.data_ptr(), w.cu.data_ptr(), w.S, w.q.shape[0], Hq, Hkv, D,
                     w.k.data_ptr(), Hkv * D, w.P, 16, w.lens.data_ptr(), *_map_args(w), w.scale, None, score.data_ptr(),
                     score.shape[1], LIMIT, s)
        assert rc == kv.OK, kv.kvsel_last_error_string(ctx.handle)
        assert kv.kvsel_check_device(ctx.handle, s) == kv.ERR_TIMEOUT, kv.kvsel_last_error_string(ctx.handle)
        call()
        ctx.check_device()
        assert torch.equal(score, want)


def test_give_up_entries_reject_bad_limits(ctx):
    import kv_cache_retention_gb300 as kv
    s = torch.cuda.current_stream().cuda_stream
    att = _entry("kvsel_test_pool_attention_give_up", "kvsel_pool_attention")
    mass = _entry("kvsel_test_attention_mass_give_up", "kvsel_attention_mass")
    for wait in (0, 2_000_000_000):
        assert att(ctx.handle, None, 128, None, 1, 1, 1, 1, 128, None, None, 128, 128, 1, 16, None, None, None, 1, -1, 1.0, None,
                   None, wait, s) == kv.ERR_INVALID_ARG
        assert mass(ctx.handle, None, 128, None, None, 1, 1, 1, 1, 128, None, 128, 1, 16, None, None, None, 1, -1, 1.0, None, None,
                    16, wait, s) == kv.ERR_INVALID_ARG
