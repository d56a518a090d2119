"""Causal attention over packed prompts with more units of work than SMs, so that every block goes through several: what
one unit loads, looks over or releases must not be taken for the next one's."""
import numpy as np
import pytest
import torch

import serving_reference as ref
from serving_reference import f64

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


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=I32).cuda()


def _inputs(lens, Hq, Hkv, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens)
    q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
    return q, k, v, np.concatenate([[0], np.cumsum(lens)])


def _run(ctx, q, k, v, cu):
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ctx.prompt_attention(q, k, v, _i32(cu), out, lse=lse)
    ctx.check_device()
    return out, lse


def _check(q, k, v, cu, out, lse, rng, per):
    """`per` random rows of each sequence and head (its first and last among them) against the formula."""
    D, G = q.shape[2], q.shape[1] // k.shape[1]
    qn, kn, vn, on, ln = f64(q), f64(k), f64(v), f64(out), f64(lse)
    scale = D ** -0.5
    for a, b in zip(cu[:-1], cu[1:]):
        for h in range(q.shape[1]):
            i = np.unique(np.concatenate([[0, b - a - 1], rng.integers(0, b - a, per)]))
            seen = np.arange(b - a)[None] <= i[:, None]
            o, l, mass, unit = ref.attention(qn[a + i, h], kn[a:b, h // G], vn[a:b, h // G], seen, scale)
            # a logit: D + 2 fp32 roundings of its absolute sum; weights rounded to bf16 (2^-8 each), exp2, sums of n
            # terms; then the output's own rounding
            n = i + 1.0
            delta = (D + 2) * 2.0 ** -24 * unit
            rel = 2.0 ** -8 + 2 * delta + (n + 16) * 2.0 ** -24
            tol = 2.0 ** -8 * np.abs(o) + rel[:, None] * mass * (1 + 2.0 ** -7) + 1e-30
            lt = delta + (n + 16) * 2.0 ** -24 + 2.0 ** -22 * np.abs(l) + 1e-6
            assert np.all(np.abs(on[a + i, h] - o) <= tol), (a, h, (np.abs(on[a + i, h] - o) / tol).max())
            assert np.all(np.abs(ln[a + i, h] - l) <= lt), (a, h, (np.abs(ln[a + i, h] - l) / lt).max())


# every unit has rows in both of its tiles
PAIRS = [256, 150, 700, 512, 129, 400, 768, 200, 255, 450, 1024, 180, 640, 500, 131, 256, 768, 390, 160, 256, 512, 250]


def _odd_values(ctx, lens, Hq, Hkv, D, seed):
    """A NaN or infinite value, and a NaN key, in every sequence: they reach the rows at and behind them, in their kv head
    and (the values) dim, and nothing else changes by a bit."""
    q, k, v, cu = _inputs(lens, Hq, Hkv, D, seed)
    clean, clean_lse = _run(ctx, q, k, v, cu)
    rng = np.random.default_rng(seed)
    _check(q, k, v, cu, clean, clean_lse, rng, 2)
    G = Hq // Hkv
    k2, v2 = k.clone(), v.clone()
    odd, gone = torch.zeros_like(clean, dtype=torch.bool), torch.zeros_like(clean, dtype=torch.bool)
    for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        h, d = int(rng.integers(Hkv)), int(rng.integers(D))
        at = int(rng.integers(max(a, b - 256), b)) if s % 3 else int(rng.integers(a, b))
        v2[at, h, d] = (float("nan"), float("inf"), -float("inf"))[s % 3]
        odd[at:b, h * G:(h + 1) * G, d] = True
        at, h = int(rng.integers(a, b)), int(rng.integers(Hkv))
        k2[at, h, int(rng.integers(D))] = float("nan")
        gone[at:b, h * G:(h + 1) * G] = True
    out, lse = _run(ctx, q, k2, v2, cu)
    assert torch.isnan(out[gone]).all() and not torch.isfinite(out[odd]).any()
    same = ~(odd | gone)
    assert torch.equal(out[same], clean[same])
    assert torch.equal(lse[~gone[..., 0]], clean_lse[~gone[..., 0]]) and torch.isnan(lse[gone[..., 0]]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,seed", [(16, 4, 1), (24, 8, 2), (16, 16, 3)])
def test_odd_values_reach_only_the_rows_that_see_them(ctx, D, Hq, Hkv, seed):
    _odd_values(ctx, PAIRS, Hq, Hkv, D, seed)


# units of one tile (up to 128 rows are left) before, between and behind units of two, and one-tile units of many keys
MIXED = [1, 300, 128, 512, 64, 257, 100, 700, 384, 2, 256, 33, 640, 127, 129, 1152, 5, 256, 1, 1, 900, 128, 400, 90, 600, 17]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,seed", [(16, 4, 4), (24, 3, 5)])
@pytest.mark.parametrize("turn", [0, 7])
def test_units_of_one_and_two_tiles_in_turn(ctx, D, Hq, Hkv, seed, turn):
    lens = MIXED[turn:] + MIXED[:turn]
    q, k, v, cu = _inputs(lens, Hq, Hkv, D, seed)
    out, lse = _run(ctx, q, k, v, cu)
    _check(q, k, v, cu, out, lse, np.random.default_rng(seed), 4)
    for _ in range(20):  # whichever block takes a unit
        again, lse2 = _run(ctx, q, k, v, cu)
        assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("D", [64, 128])
def test_odd_values_with_units_of_one_tile(ctx, D):
    _odd_values(ctx, MIXED, 16, 4, D, 6)
