"""The serving operators through the public binding against plain 64-bit implementations: slot planning, the 4-bit
cache (store, load, attention) and causal prompt attention, at the sizes and masks where they can go wrong; their
refusals; and a serving step that runs them together with the retention calls."""
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
    c.check_device()  # no test leaves an error behind
    c.close()


def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=I32).cuda()


# ---------------------------------------------------------------------------
# plan_slots
# ---------------------------------------------------------------------------

def _plan(ctx, cached, new_len, free, page, P, max_blocks, T, ld, table):
    S = len(cached)
    out = dict(table=_i32(table).reshape(S, max_blocks), cu=torch.full((S + 1,), -7, dtype=I32, device="cuda"),
               slots=torch.full((T,), -7, dtype=I32, device="cuda"), pos=torch.full((T,), -7, dtype=I32, device="cuda"),
               counts=torch.full((2,), -7, dtype=I32, device="cuda"),
               map=torch.full((S, ld), -7, dtype=I32, device="cuda") if ld else None)
    ctx.plan_slots(_i32(cached), _i32(new_len), _i32(free), page, P, out["table"], out["cu"], out["slots"], out["pos"],
                   out["counts"], slot_map=out["map"])
    return out


def _tables(rng, cached, page, max_blocks, P):
    perm = rng.permutation(P)
    table = np.full((len(cached), max_blocks), -1)
    n = 0
    for s, c in enumerate(cached):
        k = -(-c // page)
        table[s, :k] = perm[n:n + k]
        n += k
    return table, perm[n:]


@pytest.mark.parametrize("cached,new_len,page,extra,ld", [
    ([0], [1], 16, 0, 16),
    ([5], [0], 16, 0, 5),
    ([16, 0, 15, 31], [1, 0, 1, 17], 16, 3, 64),
    ([0, 0, 0], [0, 0, 0], 4, 2, 9),
    ([4095, 4096, 4097], [2, 4097, 8191], 16, 5000, 0),
    ([3, 90000, 0], [7, 2160, 1], 32, 1, 92165),
    ([1] * 700, [i % 3 for i in range(700)], 1, 11, 5),
    ([10, 7], [3, 9], 5, 0, 20),
])
def test_plan_matches_reference(ctx, cached, new_len, page, extra, ld):
    rng = np.random.default_rng(len(cached) + page)
    max_blocks = max(-(-(c + n) // page) for c, n in zip(cached, new_len)) + 1
    P = sum(-(-(c + n) // page) for c, n in zip(cached, new_len)) + 3
    table, free = _tables(rng, cached, page, max_blocks, P)
    T = sum(new_len) + extra
    got = _plan(ctx, cached, new_len, free, page, P, max_blocks, T, ld, table)
    ctx.check_device()
    want = ref.plan(cached, new_len, free, page, P, table, T, ld)
    for name, w in zip(("table", "cu", "slots", "pos", "map", "counts"), want):
        if name != "map" or ld:
            assert np.array_equal(got[name].cpu().numpy(), w), name


def test_plan_no_sessions(ctx):
    got = _plan(ctx, [], [], [], 16, 0, 1, 3, 0, np.zeros((0, 1)))
    ctx.check_device()
    assert got["cu"].tolist() == [0] and got["slots"].tolist() == [-1] * 3 and got["counts"].tolist() == [0, 0]


def _flagged(ctx, word):
    with pytest.raises(kv.KvselError, match=word):
        ctx.check_device()
    ctx.check_device()


def test_plan_too_few_free_pages(ctx):
    got = _plan(ctx, [0, 0], [20, 20], [4], 16, 8, 2, 40, 32, [[-1, -1], [-1, -1]])
    _flagged(ctx, "too few free pages")
    assert got["table"].tolist() == [[4, -1], [-1, -1]]
    assert got["slots"].tolist() == list(range(64, 80)) + [-1] * 24
    assert got["map"][0].tolist() == list(range(64, 80)) + [-1] * 16


def test_plan_lengths_out_of_range(ctx):
    # a negative length, and one past the table's row
    got = _plan(ctx, [-3, 8], [2, 100], [0, 1], 4, 4, 3, 10, 0, [[-1] * 3, [2, 3, -1]])
    _flagged(ctx, "length out of range")
    assert got["cu"].tolist() == [0, 2, 6]                     # 0 + 2 tokens; 12 positions hold 8 + 4
    assert got["table"].tolist() == [[0, -1, -1], [2, 3, 1]]
    # more tokens than new_slots holds
    got = _plan(ctx, [0], [9], [0, 1, 2], 4, 4, 3, 5, 0, [[-1] * 3])
    _flagged(ctx, "length out of range")
    assert got["slots"].tolist() == [0, 1, 2, 3, 4] and got["counts"].tolist() == [9, 3]


def test_plan_pages_of_almost_all_positions(ctx):
    """One page that takes nearly every 31-bit slot: sums next to 2^31 do not wrap."""
    page = 2 ** 31 - 4098
    table = torch.zeros((1, 1), dtype=I32, device="cuda")
    cu, slots, pos, counts = (torch.empty(n, dtype=I32, device="cuda") for n in (2, 3, 3, 2))
    ctx.plan_slots(_i32([page - 2]), _i32([2]), _i32([0]), page, 1, table, cu, slots, pos, counts)
    ctx.check_device()
    assert counts.tolist() == [2, 0] and cu.tolist() == [0, 2]  # its page is there already
    assert slots.tolist() == pos.tolist() == [page - 2, page - 1, -1]
    ctx.plan_slots(_i32([0]), _i32([2]), _i32([0]), page, 1, table, cu, slots, pos, counts)
    ctx.check_device()
    assert counts.tolist() == [2, 1] and table.tolist() == [[0]] and slots.tolist() == [0, 1, -1]


def test_plan_bad_pages(ctx):
    got = _plan(ctx, [4], [4], [9], 4, 4, 2, 4, 8, [[17, -1]])
    _flagged(ctx, "page out of range")
    assert got["table"].tolist() == [[17, -1]] and got["map"].tolist() == [[-1] * 8] and got["slots"].tolist() == [-1] * 4


# ---------------------------------------------------------------------------
# kv4_store, kv4_load
# ---------------------------------------------------------------------------

def _cache(P, Hkv, page, D, fill=0x5A):
    mk = lambda last: torch.full((P, Hkv, page, last), fill, dtype=torch.uint8, device="cuda")  # noqa: E731
    return [mk(D // 2), mk(D // 16), mk(D // 2), mk(D // 16)]


def _values(rng, T, Hkv, D):
    """Rows of mixed magnitude with zeros, signed zeros, exact ties, borders of the scale and unstorable groups."""
    x = rng.standard_normal((T, Hkv, D)) * 10.0 ** rng.uniform(-7, 4, (T, Hkv, 1))
    g = x.reshape(-1, 16)
    n = g.shape[0]
    special = [np.zeros(16), -np.zeros(16), np.r_[6.0, ref.MAGS[1:], 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25],
               np.full(16, 2.0 ** -20), np.full(16, 61440.0), np.r_[61696.0, np.ones(15)], np.r_[np.nan, np.ones(15)],
               np.r_[-np.inf, np.ones(15)], np.full(16, -6 * 2.0 ** -17), np.full(16, 1e-38)]
    for i, s in enumerate(special):
        if i < n:
            g[(i * 7) % n] = s
    for i in range(20, min(n, 247)):  # each scale's border, met exactly and just missed
        top = 6 * ref.LADDER[i - 20]
        g[i, 3] = top if i % 2 else top * (1 + 2.0 ** -7)
        g[i, 4:] = np.clip(g[i, 4:], -top, top)
    return x


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("T,Hkv,D,page", [(1, 1, 64, 1), (37, 2, 128, 16), (5, 8, 256, 7), (131, 3, 64, 64)])
def test_store_and_load_exact(ctx, dtype, T, Hkv, D, page):
    rng = np.random.default_rng(T + D)
    k = torch.from_numpy(_values(rng, T, Hkv, D)).to(dtype).cuda()
    v = torch.from_numpy(_values(rng, T, Hkv, D)[::-1].copy()).to(dtype).cuda()
    P = -(-T // page) + 2
    slots = rng.permutation(P * page)[:T]
    if T > 4:
        slots[3] = -1
    cache = _cache(P, Hkv, page, D)
    ctx.kv4_store(k, v, _i32(slots), *cache)
    kb, vb = torch.full_like(k, 7, dtype=BF), torch.full_like(v, 7, dtype=BF)
    ctx.kv4_load(*cache, _i32(slots), kb, vb)
    ctx.check_device()
    got = [c.cpu().numpy() for c in cache]
    for x, back, codes, scales in ((k, kb, got[0], got[1]), (v, vb, got[2], got[3])):
        rc, rs = ref.quantise(f64(x))
        want = ref.dequantise(rc, rs)
        written = np.zeros((P, page), bool)
        for i, slot in enumerate(slots):
            if slot < 0:
                assert not back[i].any()
                continue
            written[slot // page, slot % page] = True
            assert np.array_equal(codes[slot // page, :, slot % page], rc[i])
            assert np.array_equal(scales[slot // page, :, slot % page], rs[i])
            assert np.array_equal(f64(back[i]), want[i], equal_nan=True)
        rest = ~written[:, None, :, None]
        assert np.all(codes[np.broadcast_to(rest, codes.shape)] == 0x5A)
        assert np.all(scales[np.broadcast_to(rest, scales.shape)] == 0x5A)


def test_store_rounds_fp32_next_to_ties(ctx):
    """fp32 values one step to each side of every border, for every scale mantissa."""
    rows = []
    for m in range(8):
        s = np.float32((1 + m / 8) * 4)
        for b in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
            t = np.float32(b) * s
            rows.append([6 * s, t, np.nextafter(t, np.float32(0)), np.nextafter(t, np.float32(1e9))] + [0] * 12)
    x = torch.tensor(np.array(rows, np.float32).reshape(-1, 1, 64)).cuda()
    T = x.shape[0]
    cache = _cache(T, 1, 1, 64)
    ctx.kv4_store(x, x, torch.arange(T, dtype=I32, device="cuda"), *cache)
    ctx.check_device()
    rc, rs = ref.quantise(f64(x))
    assert np.array_equal(cache[0].cpu().numpy()[:, 0, 0], rc[:, 0]) and np.array_equal(cache[3].cpu().numpy()[:, 0, 0], rs[:, 0])


def test_store_strided_rows_and_every_bf16(ctx):
    """Slices of a fused projection as sources; all finite bf16 values as group members."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF)
    bits = bits[bits.abs() <= 61440.0]
    bits = bits[: bits.numel() // 1024 * 1024].reshape(-1, 4, 128).cuda()  # neighbours share a group
    T = bits.shape[0]
    fused = torch.zeros((T, 8 + 4 + 4, 128), dtype=BF, device="cuda")
    fused[:, 8:12], fused[:, 12:] = bits, bits.flip(0)
    cache = _cache(T // 16 + 1, 4, 16, 128)
    slots = torch.arange(T, dtype=I32, device="cuda").flip(0).contiguous()
    ctx.kv4_store(fused[:, 8:12], fused[:, 12:], slots, *cache)
    back = torch.zeros((T, 8, 128), dtype=BF, device="cuda")
    ctx.kv4_load(*cache, slots, back[:, :4], back[:, 4:])
    ctx.check_device()
    for x, b in ((bits, back[:, :4]), (bits.flip(0), back[:, 4:])):
        assert np.array_equal(f64(b), ref.dequantise(*ref.quantise(f64(x))))


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("T", [5, 6001])
def test_store_and_load_rows_on_16_bytes(ctx, dtype, T):
    """Rows that lie on 16 bytes and not on 32 (K's, V's or both), few tokens and many, are stored like others."""
    g = torch.Generator(device="cuda").manual_seed(T)
    Hkv, D, page = 8, 64, 16
    k, v = (torch.randn((T, Hkv, D), generator=g, device="cuda").to(dtype) for _ in range(2))
    step = 16 // k.element_size()
    slots = torch.randperm(T + 30, generator=g, device="cuda")[:T].to(I32)
    P = (T + 30 + page - 1) // page

    def shifted(x, by):
        y = torch.zeros(x.numel() + by, dtype=x.dtype, device="cuda")[by:].view(x.shape)
        return y.copy_(x)

    want = _cache(P, Hkv, page, D)
    ctx.kv4_store(k, v, slots, *want)
    first = torch.randint(0, T, (5,), generator=g, device="cuda").tolist()
    for i in first:
        rc, rs = ref.quantise(f64(k[i]))
        n = int(slots[i])
        assert np.array_equal(want[0][n // page, :, n % page].cpu().numpy(), rc)
        assert np.array_equal(want[1][n // page, :, n % page].cpu().numpy(), rs)
    kb, vb = torch.empty((T, Hkv, D), dtype=BF, device="cuda"), torch.empty((T, Hkv, D), dtype=BF, device="cuda")
    ctx.kv4_load(*want, slots, kb, vb)
    for bk, bv in ((step, 0), (0, step), (step, step)):
        got = _cache(P, Hkv, page, D)
        ctx.kv4_store(shifted(k, bk), shifted(v, bv), slots, *got)
        assert all(torch.equal(i, j) for i, j in zip(got, want))
        ko, vo = shifted(torch.zeros_like(kb), bk and 8), shifted(torch.zeros_like(vb), bv and 8)
        ctx.kv4_load(*want, slots, ko, vo)
        assert torch.equal(ko, kb) and torch.equal(vo, vb)
    ctx.check_device()


def test_every_code_and_scale_loads_exactly(ctx):
    codes = np.arange(256, dtype=np.uint8).reshape(4, 64)[None].repeat(256, 0).reshape(1024, 1, 1, 64)
    scales = np.repeat(np.arange(256, dtype=np.uint8), 4)[:, None].repeat(8, 1).reshape(1024, 1, 1, 8)
    scales[scales > 226] = 255  # the format's bytes: up to 226, and 255
    c, s = ref.torch_u8(codes), ref.torch_u8(scales)
    k, v = torch.empty((1024, 1, 128), dtype=BF, device="cuda"), torch.empty((1024, 1, 128), dtype=BF, device="cuda")
    ctx.kv4_load(c, s, c, s, torch.arange(1024, dtype=I32, device="cuda"), k, v)
    ctx.check_device()
    want = ref.dequantise(codes, scales)[:, 0]
    assert np.array_equal(f64(k), want, equal_nan=True) and np.array_equal(f64(v), want, equal_nan=True)


def test_store_slots_out_of_range(ctx):
    x = torch.ones((3, 1, 64), dtype=BF, device="cuda")
    cache = _cache(2, 1, 4, 64)
    before = [c.clone() for c in cache]
    ctx.kv4_store(x, x, _i32([8, 2 ** 31 - 1, -2 ** 31]), *cache)
    _flagged(ctx, "slot out of range")
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    out = torch.full_like(x, 3)
    ctx.kv4_load(*cache, _i32([8, -1, 2 ** 31 - 1]), out, out.clone())
    _flagged(ctx, "slot out of range")
    assert not out.any()


# ---------------------------------------------------------------------------
# kv4_attention
# ---------------------------------------------------------------------------

def _random_cache(g, P, Hkv, page, D, lo=100, hi=124):
    """Random codes and scales (2^-2.5 .. 2^0.5 by default) and NaN groups nowhere."""
    codes = lambda: torch.randint(0, 256, (P, Hkv, page, D // 2), generator=g, device="cuda").to(torch.uint8)  # noqa: E731
    scales = lambda: torch.randint(lo, hi, (P, Hkv, page, D // 16), generator=g, device="cuda").to(torch.uint8)  # noqa: E731
    return [codes(), scales(), codes(), scales()]


def _attention_reference(q, cache, lens, slots, live, scale):
    """slots, live [S][reach] (numpy) -> out, lse and their tolerances."""
    q = f64(q)
    kc, ks, vc, vs = (c.cpu().numpy() for c in cache)
    P, Hkv, page, _ = kc.shape
    S, Tq, Hq, D = q.shape
    G = Hq // Hkv
    out, lse = np.zeros(q.shape), np.full((S, Tq, Hq), -np.inf)
    out_tol, lse_tol = np.zeros(q.shape), np.zeros((S, Tq, Hq))
    for s in range(S):
        j = np.flatnonzero(live[s, :max(0, lens[s])])
        sl = slots[s, j]
        for h in range(Hkv):
            k = ref.dequantise(kc[sl // page, h, sl % page], ks[sl // page, h, sl % page])
            v = ref.dequantise(vc[sl // page, h, sl % page], vs[sl // page, h, sl % page])
            rows = q[s, :, h * G:(h + 1) * G].reshape(Tq * G, D)
            seen = np.repeat(j[None] <= (lens[s] - Tq + np.arange(Tq))[:, None], G, 0)
            o, l, mass, unit = ref.attention(rows, k, v, seen, scale)
            # a logit: D+2 fp32 roundings of its absolute sum, and the query rows' fp16 underflow (2^-25 of the row's
            # largest value a product); a weight: fp16 (2^-11), exp2 and the sums over n tokens (2^-24 each)
            n = max(1, len(j))
            peak = np.abs(rows).max(-1) * scale * (np.abs(k).sum(-1).max() if len(j) else 0)
            delta = (D + 2) * 2.0 ** -24 * unit + 2.0 ** -25 * peak
            rel = 2.0 ** -11 + 2 * delta + (n + 16) * 2.0 ** -24
            # fp16 holds weights as multiples of 2^-24 at least, with the row's largest weight at 2^10 or above: one of
            # them is off by up to 2^-25 / 2^10 of the largest, which the sum of the weights is not below
            lost = np.stack([2.0 ** -35 * np.abs(v[sn]).sum(0) for sn in seen])
            ot = 2.0 ** -8 * np.abs(o) + rel[:, None] * mass * (1 + 2.0 ** -7) + lost * (1 + 2.0 ** -7) + 1e-30
            lt = delta + (n + 16) * 2.0 ** -24 + 2.0 ** -22 * np.where(np.isinf(l), 0, np.abs(l)) + 1e-6
            put = lambda a, b: a.__setitem__((s, slice(None), slice(h * G, (h + 1) * G)), b)  # noqa: E731
            put(out, o.reshape(Tq, G, D)), put(out_tol, ot.reshape(Tq, G, D))
            put(lse, l.reshape(Tq, G)), put(lse_tol, lt.reshape(Tq, G))
    return out, lse, out_tol, lse_tol


def _check_attention(got, got_lse, want):
    out, lse, out_tol, lse_tol = want
    got, got_lse = f64(got), f64(got_lse)
    assert np.array_equal(np.isinf(got_lse), np.isinf(lse)) and not np.isnan(got_lse).any()
    fin = ~np.isinf(lse)
    assert np.all(np.abs(got_lse[fin] - lse[fin]) <= lse_tol[fin]), np.abs(got_lse[fin] - lse[fin]).max()
    assert np.all(np.abs(got - out) <= out_tol), (np.abs(got - out) / out_tol).max()
    assert not got[np.isinf(lse)].any()


ATTENTION = [
    # S, Tq, Hq, Hkv, D, page, lens
    (1, 1, 1, 1, 64, 1, [1]),
    (1, 1, 4, 2, 64, 16, [31]),
    (2, 1, 8, 1, 128, 16, [0, 33]),
    (3, 1, 10, 2, 128, 32, [257, 64, 1]),
    (4, 1, 32, 8, 128, 16, [700, 5, 513, 0]),
    (2, 4, 8, 2, 128, 16, [2, 130]),       # fewer tokens than query rows: the first rows see nothing
    (2, 7, 6, 2, 64, 7, [100, 61]),
    (1, 3, 16, 1, 256, 16, [95]),
    (2, 1, 12, 1, 256, 3, [45, 200]),      # groups of twelve heads
    (1, 40, 8, 2, 128, 16, [300]),         # a short continuation
    (1, 1, 5, 1, 128, 64, [5000]),
    (2, 130, 16, 8, 64, 16, [150, 131]),   # more row tiles than the GPU takes blocks at a time
    (1, 600, 12, 12, 64, 8, [601]),
    (7, 1, 4, 2, 64, 16, [2000, 3, 900, 0, 1, 31, 4097]),
    (40, 2, 8, 2, 64, 16, [1 + 37 * i for i in range(40)]),
    (600, 1, 1, 1, 64, 16, [i % 70 for i in range(600)]),
    (300, 1, 2, 1, 64, 16, [(i * i * 37) % 900 for i in range(299)] + [2500]),
    (9, 3, 8, 4, 128, 16, [2100, 0, 1, 2100, 40, 0, 1000, 3, 2222]),
    (40, 1, 16, 8, 128, 16, [1 + 50 * i for i in range(40)]),
    (40, 1, 16, 8, 128, 16, [1 + 25 * i for i in range(40)]),           # sessions of their own blocks, up to 1024
    (3, 1, 2, 1, 128, 16, [767, 768, 769]),
    (2, 1, 4, 2, 128, 48, [1500, 950]),
    (160, 1, 4, 2, 64, 16, [(i * 397) % 2040 for i in range(160)]),
    (160, 1, 4, 2, 64, 16, [(i * 397) % 990 for i in range(160)]),
]


@pytest.mark.parametrize("S,Tq,Hq,Hkv,D,page,lens", ATTENTION)
@pytest.mark.parametrize("kind", ["table", "map"])
def test_attention_matches_reference(ctx, S, Tq, Hq, Hkv, D, page, lens, kind):
    g = torch.Generator(device="cuda").manual_seed(S * 1000 + D + Hq)
    rng = np.random.default_rng(D + Hq)
    rows = -(-max(lens + [1]) // page) + 1
    P = S * rows
    cache = _random_cache(g, P, Hkv, page, D)
    q = torch.randn((S, Tq, Hq, D), generator=g, device="cuda").to(BF)
    table = rng.permutation(P).reshape(S, rows)
    j = np.arange(rows * page)
    slots = table[:, j // page] * page + j % page
    live = np.ones_like(slots, bool)
    args = dict(block_table=_i32(table))
    if kind == "map":  # some tokens dropped to the dead slot, some to -1; what lies behind the length is not looked at
        drop = rng.random(slots.shape)
        live = drop > 0.4
        sm = np.where(drop < 0.2, P * page, np.where(live, slots, -1))
        sm[j[None] >= np.array(lens)[:, None]] = 2 ** 31 - 1
        args = dict(slot_map=_i32(sm), dead_slot=P * page)
    out, lse = torch.full_like(q, 9), torch.full((S, Tq, Hq), 9.0, device="cuda")
    ctx.kv4_attention(q, *cache, _i32(lens), out, lse=lse, **args)
    ctx.check_device()
    _check_attention(out, lse, _attention_reference(q, cache, lens, slots, live, D ** -0.5))


def test_attention_never_reads_dropped_rows(ctx):
    """NaN groups in dropped rows, in rows behind the length and in other sessions' pages change nothing."""
    g = torch.Generator(device="cuda").manual_seed(5)
    S, Hq, Hkv, D, page, N = 2, 8, 2, 128, 16, 200
    cache = _random_cache(g, 30, Hkv, page, D)
    q = torch.randn((S, 1, Hq, D), generator=g, device="cuda").to(BF)
    rng = np.random.default_rng(1)
    slots = np.stack([rng.permutation(30 * page)[:N] for _ in range(S)])
    live = rng.random((S, N)) < 0.5
    lens = [200, 120]
    live[0, :], live[0, 77] = False, True  # one live token of 200
    used = np.zeros(30 * page, bool)
    for s in range(S):
        used[slots[s, :lens[s]][live[s, :lens[s]]]] = True
    flat = torch.from_numpy(~used).cuda().view(30, 1, page, 1)
    for i in (1, 3):
        cache[i].masked_fill_(flat, 255)
    dead = 30 * page
    sm = np.where(live, slots, dead)
    out, lse = torch.empty_like(q), torch.empty((S, 1, Hq), device="cuda")
    ctx.kv4_attention(q, *cache, _i32(lens), out, slot_map=_i32(sm), dead_slot=dead, lse=lse)
    ctx.check_device()
    _check_attention(out, lse, _attention_reference(q, cache, lens, slots, live, D ** -0.5))
    # a NaN group that is seen comes out
    cache[3].view(-1, 8)[:] = 255
    ctx.kv4_attention(q, *cache, _i32(lens), out, slot_map=_i32(sm), dead_slot=dead, lse=lse)
    ctx.check_device()
    assert torch.isnan(out).all()


@pytest.mark.parametrize("Tq", [1, 3])
def test_attention_nan_keys_and_queries(ctx, Tq):
    """A NaN key group makes the rows that see it NaN, a NaN query its own row, in one kv head only; the rows before
    the token stay as they are, also where it is the only thing a warp sees."""
    g = torch.Generator(device="cuda").manual_seed(15)
    Hq, Hkv, D, page, n = 8, 2, 128, 16, 77
    cache = _random_cache(g, 5, Hkv, page, D)
    q = torch.randn((1, Tq, Hq, D), generator=g, device="cuda").to(BF)
    table = _i32([[3, 0, 4, 1, 2]])
    clean = torch.empty_like(q)
    ctx.kv4_attention(q, *cache, _i32([n]), clean, block_table=table)
    bad = [c.clone() for c in cache]
    bad[1][2, 0, (n - 1) % page, 2] = 255               # the last token's key, kv head 0
    bad[3][2, 1, (n - 1) % page, 4] = 255               # and its value, kv head 1
    out, lse = torch.empty_like(q), torch.empty((1, Tq, Hq), device="cuda")
    ctx.kv4_attention(q, *bad, _i32([n]), out, block_table=table, lse=lse)
    assert torch.equal(out[:, :-1], clean[:, :-1])
    assert torch.isnan(out[0, -1, :4]).all() and torch.isnan(lse[0, -1, :4]).all()
    assert torch.isnan(out[0, -1, 4:, 64:80]).all() and torch.isfinite(lse[0, -1, 4:]).all()
    keep = torch.ones(D, dtype=torch.bool, device="cuda")
    keep[64:80] = False
    assert torch.equal(out[0, -1, 4:, keep], clean[0, -1, 4:, keep])
    q2 = q.clone()
    q2[0, 0, 1, 9] = float("nan")
    bad[1].fill_(255)
    ctx.kv4_attention(q2, *cache, _i32([n]), out, block_table=table, lse=lse)
    assert torch.isnan(out[0, 0, 1]).all() and torch.isnan(lse[0, 0, 1])
    out[0, 0, 1] = clean[0, 0, 1]
    assert torch.equal(out, clean)
    ctx.kv4_attention(q, *bad, _i32([n]), out, block_table=table, lse=lse)  # nothing but NaN keys
    ctx.check_device()
    assert torch.isnan(out).all() and torch.isnan(lse).all()


def test_attention_dead_slot_inside_the_pool(ctx):
    """The dead slot may be a real row of the pool: it is skipped all the same."""
    g = torch.Generator(device="cuda").manual_seed(6)
    cache = _random_cache(g, 4, 1, 16, 64)
    q = torch.randn((1, 1, 4, 64), generator=g, device="cuda").to(BF)
    slots = np.arange(64)[None]
    sm = np.where(np.arange(64) % 3 == 0, 9, np.arange(64))[None]
    live = sm != 9
    out, lse = torch.empty_like(q), torch.empty((1, 1, 4), device="cuda")
    ctx.kv4_attention(q, *cache, _i32([64]), out, slot_map=_i32(sm), dead_slot=9, lse=lse)
    ctx.check_device()
    _check_attention(out, lse, _attention_reference(q, cache, [64], slots, live, 64 ** -0.5))


@pytest.mark.parametrize("qs,lo,hi,scale", [(1.0, 0, 8, 1.0), (2.0 ** 60, 1, 9, 2.0 ** -60), (2.0 ** -60, 200, 227, 2.0 ** 50),
                                            (300.0, 100, 124, 1.0), (1e-30, 100, 124, 1.0)])
def test_attention_extreme_values(ctx, qs, lo, hi, scale):
    """Subnormal and largest scales, query rows far outside fp16, logits of thousands and of nothing."""
    g = torch.Generator(device="cuda").manual_seed(hi)
    cache = _random_cache(g, 8, 2, 16, 128, lo, hi)
    q = (torch.randn((1, 2, 8, 128), generator=g, device="cuda") * qs).to(BF)
    q[0, 0, 1] = 0  # a row of zeros: the mean
    q[0, 1, 2, 5:] = 0
    table = np.arange(8)[None]
    out, lse = torch.empty_like(q), torch.empty((1, 2, 8), device="cuda")
    ctx.kv4_attention(q, *cache, _i32([125]), out, block_table=_i32(table), lse=lse, scale=scale)
    ctx.check_device()
    _check_attention(out, lse, _attention_reference(q, cache, [125], np.arange(128)[None], np.ones((1, 128), bool), scale))


def test_attention_bad_lengths_slots_and_pages(ctx):
    g = torch.Generator(device="cuda").manual_seed(8)
    cache = _random_cache(g, 4, 1, 16, 64)
    q = torch.randn((2, 1, 4, 64), generator=g, device="cuda").to(BF)
    out, lse = torch.empty_like(q), torch.empty((2, 1, 4), device="cuda")
    table = np.array([[0, 1], [2, 3]])
    j = np.arange(32)
    slots = table[:, j // 16] * 16 + j % 16
    every = np.ones((2, 32), bool)
    ctx.kv4_attention(q, *cache, _i32([33, -1]), out, block_table=_i32(table), lse=lse)
    _flagged(ctx, "length out of range")
    _check_attention(out, lse, _attention_reference(q, cache, [32, 0], slots, every, 0.125))
    bad = table.copy()
    bad[0, 1], bad[1, 0] = 4, -1
    live = every.copy()
    live[0, 16:], live[1, :16] = False, False
    ctx.kv4_attention(q, *cache, _i32([32, 32]), out, block_table=_i32(bad), lse=lse)
    _flagged(ctx, "page out of range")
    _check_attention(out, lse, _attention_reference(q, cache, [32, 32], slots, live, 0.125))
    sm = slots.copy()
    sm[0, 3], sm[1, 31] = 64, 2 ** 31 - 1
    live = every.copy()
    live[0, 3], live[1, 31] = False, False
    ctx.kv4_attention(q, *cache, _i32([32, 32]), out, slot_map=_i32(sm), lse=lse)
    _flagged(ctx, "slot out of range")
    _check_attention(out, lse, _attention_reference(q, cache, [32, 32], slots, live, 0.125))


def test_attention_strided_queries_and_no_lse(ctx):
    g = torch.Generator(device="cuda").manual_seed(9)
    S, Tq, Hq, Hkv, D = 3, 2, 6, 2, 128
    cache = _random_cache(g, 12, Hkv, 16, D)
    fused = torch.randn((S, Tq, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
    table = np.arange(12).reshape(3, 4)
    a, b = torch.empty((S, Tq, Hq, D), dtype=BF, device="cuda"), torch.empty((S, Tq, Hq, D), dtype=BF, device="cuda")
    lens = _i32([64, 17, 40])
    ctx.kv4_attention(fused[:, :, :Hq], *cache, lens, a, block_table=_i32(table))
    ctx.kv4_attention(fused[:, :, :Hq].contiguous(), *cache, lens, b, block_table=_i32(table))
    ctx.check_device()
    assert torch.equal(a, b)


def test_attention_long_cache_past_32_bits(ctx):
    """A pool whose byte offsets pass 2^32: rows at its end are read where they are."""
    D, Hkv, page = 128, 8, 32
    P = (1 << 32) // (Hkv * page * D // 2) + 40
    g = torch.Generator(device="cuda").manual_seed(10)
    big = [torch.zeros((P, Hkv, page, last), dtype=torch.uint8, device="cuda") for last in (64, 8, 64, 8)]
    small = _random_cache(g, 40, Hkv, page, D)
    for b, s in zip(big, small):
        b[P - 40:] = s
    q = torch.randn((1, 1, 32, D), generator=g, device="cuda").to(BF)
    table = torch.arange(40, dtype=I32, device="cuda")[None].contiguous()
    outs = [torch.empty_like(q) for _ in range(2)]
    n = _i32([40 * page - 3])
    ctx.kv4_attention(q, *big, n, outs[0], block_table=table + (P - 40))
    ctx.kv4_attention(q, *small, n, outs[1], block_table=table)
    x = torch.randn((2, Hkv, D), generator=g, device="cuda").to(BF)
    last = _i32([P * page - 1, (P - 1) * page])
    ctx.kv4_store(x, x, last, *big)
    back = [torch.empty_like(x) for _ in range(2)]
    ctx.kv4_load(*big, last, *back)
    ctx.check_device()
    assert torch.equal(*outs)
    assert np.array_equal(f64(back[0]), ref.dequantise(*ref.quantise(f64(x))))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_over_runs_of_slots(ctx, D):
    """Maps of consecutive slots that start anywhere, whole and with gaps: taken by bulk copies or one by one."""
    g = torch.Generator(device="cuda").manual_seed(D)
    S, Hq, Hkv, P, page = 7, 4, 2, 2, 1024
    cache = _random_cache(g, P, Hkv, page, D)
    q = torch.randn((S, 2, Hq, D), generator=g, device="cuda").to(BF)
    j = np.arange(640)
    slots = np.stack([j + 5 * 64 + s for s in range(S)])  # across the pages' border, at starts of every alignment
    live = np.ones_like(slots, bool)
    live[5, 100:103] = live[6, ::5] = False
    lens = [640, 639, 500, 33, 600, 640, 640]
    out, lse = torch.empty_like(q), torch.empty((S, 2, Hq), device="cuda")
    ctx.kv4_attention(q, *cache, _i32(lens), out, slot_map=_i32(np.where(live, slots, -1)), lse=lse)
    ctx.check_device()
    _check_attention(out, lse, _attention_reference(q, cache, lens, slots, live, D ** -0.5))


def test_attention_graphs_in_turn(ctx):
    """Two captured calls of one context (shared partial results), replayed in turn with eager calls between them."""
    g = torch.Generator(device="cuda").manual_seed(31)
    cases = []
    for S, Tq, Hq, Hkv, D, n in ((2, 1, 8, 2, 128, 4000), (5, 3, 6, 1, 64, 2500)):
        rows = n // 16 + 1
        cache = _random_cache(g, S * rows, Hkv, 16, D)
        table = torch.randperm(S * rows, generator=g, device="cuda").to(I32).view(S, rows).contiguous()
        q = torch.randn((S, Tq, Hq, D), generator=g, device="cuda").to(BF)
        lens = torch.randint(n // 2, n, (S,), generator=g, device="cuda").to(I32)
        out, lse = torch.empty_like(q), torch.empty((S, Tq, Hq), device="cuda")
        call = lambda q=q, cache=cache, lens=lens, out=out, table=table, lse=lse: ctx.kv4_attention(  # noqa: E731
            q, *cache, lens, out, block_table=table, lse=lse)
        call()
        torch.cuda.synchronize()
        want = out.clone(), lse.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        cases.append((graph, call, out, lse, want))
    for i in range(6):
        for graph, call, out, lse, want in cases:
            out.fill_(7), lse.fill_(7)
            graph.replay() if (i + (out is cases[0][2])) % 3 else call()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    ctx.check_device()


def test_attention_is_deterministic(ctx):
    g = torch.Generator(device="cuda").manual_seed(11)
    cache = _random_cache(g, 512, 2, 16, 128)
    q = torch.randn((3, 1, 8, 128), generator=g, device="cuda").to(BF)
    table = torch.randperm(512, generator=g, device="cuda").to(I32)[:510].view(3, 170).contiguous()
    lens = _i32([2711, 900, 2720])
    outs = []
    for _ in range(5):
        o, l = torch.empty_like(q), torch.empty((3, 1, 8), device="cuda")
        ctx.kv4_attention(q, *cache, lens, o, block_table=table, lse=l)
        outs.append((o, l))
    ctx.check_device()
    assert all(torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1]) for o, l in outs)


# ---------------------------------------------------------------------------
# prompt_attention
# ---------------------------------------------------------------------------

def _check_prompt(q, k, v, cu, scale, out, lse, rows=None):
    """Rows (all, or the given tokens) against the formula; bf16 weights, fp32 sums."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    qn, kn, vn, on, ln = f64(q), f64(k), f64(v), f64(out), None if lse is None else f64(lse)
    for a, b in zip(cu[:-1], cu[1:]):
        at = np.arange(a, b) if rows is None else np.array([r for r in rows if a <= r < b], int)
        if not at.size:
            continue
        for h in range(Hq):
            kk, vv = kn[a:b, h // G], vn[a:b, h // G]
            seen = np.arange(b - a)[None] <= (at - a)[:, None]
            o, l, mass, unit = ref.attention(qn[at, h], kk, vv, seen, scale)
            n = (at - a + 1).astype(float)
            delta = (D + 2) * 2.0 ** -24 * unit
            # weights rounded to bf16 (2^-8 each), exp2, sums of n terms; then the output's own rounding
            rel = 2.0 ** -8 + 2 * delta + (n + 16) * 2.0 ** -24
            tol = 2.0 ** -8 * np.abs(o) + rel[:, None] * mass * (1 + 2.0 ** -7) + 1e-30
            assert np.all(np.abs(on[at, h] - o) <= tol), (h, (np.abs(on[at, h] - o) / tol).max())
            if ln is not None:
                lt = delta + (n + 16) * 2.0 ** -24 + 2.0 ** -22 * np.abs(l) + 1e-6
                assert np.all(np.abs(ln[at, h] - l) <= lt), (h, (np.abs(ln[at, h] - l) / lt).max())


PROMPT = [
    # lengths, Hq, Hkv, D
    ([1], 1, 1, 64),
    ([1], 4, 2, 128),
    ([2, 0, 1], 2, 1, 128),
    ([127], 4, 2, 64),
    ([128], 2, 2, 128),
    ([129, 1, 255], 8, 2, 128),
    ([256, 257], 5, 1, 128),
    ([513], 6, 2, 64),
    ([0, 0, 300, 0], 3, 3, 128),
    ([1] * 70, 2, 1, 128),
    ([640, 3, 77, 129], 16, 2, 64),
    ([1100], 10, 2, 128),
    ([700, 0, 128, 257], 9, 3, 64),        # units of one tile of 128 rows, and with more heads of two
    ([700, 0, 128, 256, 1], 16, 4, 64),
]


@pytest.mark.parametrize("lens,Hq,Hkv,D", PROMPT)
@pytest.mark.parametrize("fused", [False, True])
def test_prompt_matches_reference(ctx, lens, Hq, Hkv, D, fused):
    T = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(T + Hq)
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    cu = np.concatenate([[0], np.cumsum(lens)])
    out, lse = torch.full((T, Hq, D), 9.0, dtype=BF, device="cuda"), torch.full((T, Hq), 9.0, device="cuda")
    ctx.prompt_attention(q, k, v, _i32(cu), out, lse=lse)
    ctx.check_device()
    _check_prompt(q, k, v, cu, D ** -0.5, out, lse)


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (40, 4)])
def test_prompt_rows_outside_sequences_stay(ctx, Hq, Hkv):
    """A gap before the first sequence and padding behind the last: outputs there are left, and NaN inputs there and in
    later tokens reach no row."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, D = 400, 128
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
    qkv[:7] = float("nan")
    qkv[330:] = float("inf")
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cu = [7, 150, 330]
    out, lse = torch.full((T, Hq, D), 9.0, dtype=BF, device="cuda"), torch.full((T, Hq), 9.0, device="cuda")
    ctx.prompt_attention(q, k, v, _i32(cu), out, lse=lse)
    ctx.check_device()
    for x in (out, lse):
        assert (x[:7] == 9).all() and (x[330:] == 9).all() and torch.isfinite(x[7:330].float()).all()
    _check_prompt(q, k, v, cu, D ** -0.5, out, lse)


@pytest.mark.parametrize("H", [2, 50])
def test_prompt_future_nan_is_not_seen(ctx, H):
    """A NaN or infinite key or value reaches the rows at and behind it, and none before it (same tile)."""
    g = torch.Generator(device="cuda").manual_seed(4)
    T, D = 300, 128
    q, k, v = (torch.randn((T, H, D), generator=g, device="cuda").to(BF) for _ in range(3))
    for bad in (float("nan"), float("inf")):
        k2, v2 = k.clone(), v.clone()
        k2[141, 0, 5], v2[205, 1, 7] = float("nan"), bad
        out = torch.empty_like(q)
        ctx.prompt_attention(q, k2, v2, _i32([0, T]), out)
        ctx.check_device()
        clean = torch.empty_like(q)
        ctx.prompt_attention(q, k, v, _i32([0, T]), clean)
        assert torch.equal(out[:141, 0], clean[:141, 0]) and torch.isnan(out[141:, 0]).all()
        assert torch.equal(out[:205, 1], clean[:205, 1]) and not torch.isfinite(out[205:, 1, 7]).any()


@pytest.mark.parametrize("qs,scale", [(1.0, 20.0), (60.0, 1.0), (1e-20, 1.0), (2.0 ** 50, 2.0 ** -50)])
@pytest.mark.parametrize("H", [2, 30])
def test_prompt_extreme_logits(ctx, H, qs, scale):
    """Logits of thousands (one weight near 1), rising along the sequence, and of nothing (the mean)."""
    g = torch.Generator(device="cuda").manual_seed(13)
    T, D = 700, 64
    q, k, v = (torch.randn((T, H, D), generator=g, device="cuda") for _ in range(3))
    q = (q * qs).to(BF)
    k = (k * torch.linspace(0.1, 3, T, device="cuda")[:, None, None]).to(BF)
    v = v.to(BF)
    out, lse = torch.empty_like(v), torch.empty((T, H), device="cuda")
    ctx.prompt_attention(q, k, v, _i32([0, T]), out, lse=lse, scale=scale)
    ctx.check_device()
    _check_prompt(q, k, v, [0, T], scale, out, lse)


def test_prompt_long_sampled_rows(ctx):
    g = torch.Generator(device="cuda").manual_seed(14)
    lens = [9000, 513]
    T, Hq, Hkv, D = sum(lens), 8, 2, 128
    q = torch.randn((T, Hq, D), generator=g, device="cuda").to(BF)
    k, v = (torch.randn((T, Hkv, D), generator=g, device="cuda").to(BF) for _ in range(2))
    out, lse = torch.empty_like(q), torch.empty((T, Hq), device="cuda")
    ctx.prompt_attention(q, k, v, _i32([0, 9000, T]), out, lse=lse)
    ctx.check_device()
    _check_prompt(q, k, v, [0, 9000, T], D ** -0.5, out, lse, rows=[0, 1, 127, 128, 4095, 4096, 8191, 8999, 9000, 9127, T - 1])


def test_prompt_bad_starts_are_flagged(ctx):
    x = torch.ones((8, 1, 64), dtype=BF, device="cuda")
    out = torch.full_like(x, 9)
    ctx.prompt_attention(x, x, x, _i32([-4, 8]), out)
    _flagged(ctx, "length out of range")
    assert (out == 9).all()


@pytest.mark.parametrize("cu", [[0, 9], [5, -2 ** 31], [2 ** 31 - 1, 2 ** 31 - 1], [3, 2, 8], [-2 ** 31, 2 ** 31 - 1],
                                [0, 2 ** 31 - 1, 8], [600, 700], [0, 300, 100, 8]])
def test_prompt_bad_sequences_are_flagged(ctx, cu):
    """Sequences outside the rows, or descending: flagged, and nothing outside the rows is written."""
    T = 8
    big = torch.ones((1024, 2, 64), dtype=BF, device="cuda")
    out, lse = torch.full_like(big, 9), torch.full((1024, 2), 9.0, device="cuda")
    ctx.prompt_attention(big[:T], big[:T], big[:T], _i32(cu), out[:T], lse=lse[:T])
    _flagged(ctx, "length out of range")
    assert (out[T:] == 9).all() and (lse[T:] == 9).all()


@pytest.mark.parametrize("H", [1, 50])
def test_prompt_minus_infinite_logits_of_the_last_keys(ctx, H):
    """Keys whose logits are -inf for every row: a softmax over the keys before them, as the formula has it."""
    g = torch.Generator(device="cuda").manual_seed(23)
    T, D, cut = 300, 64, 200
    q, k, v = (torch.randn((T, H, D), generator=g, device="cuda").to(BF) for _ in range(3))
    q[..., 0] = 1
    k[cut:, :, 0] = -float("inf")
    q[..., 1] = q[..., 1].abs() + 1
    k[:cut, :, 1] = -200  # far below zero where they are finite: logits near -25 to -100
    out, lse = torch.empty_like(q), torch.empty((T, H), device="cuda")
    ctx.prompt_attention(q, k, v, _i32([0, T]), out, lse=lse)
    ctx.check_device()
    # rows before the cut as they are; each later row like one that sees the first `cut` keys
    _check_prompt(q[:cut], k[:cut], v[:cut], [0, cut], D ** -0.5, out[:cut], lse[:cut])
    for r in (cut, 255, 256, 299):
        at = [r if i == cut - 1 else i for i in range(cut)]
        _check_prompt(q[at], k[:cut], v[:cut], [0, cut], D ** -0.5, out[at], lse[at], rows=[cut - 1])


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def test_refusals(ctx):
    h, s = ctx.handle, torch.cuda.current_stream().cuda_stream
    x = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = x.data_ptr()
    att = lambda **kw: kv.kvsel_kv4_attention(*{**dict(  # noqa: E731
        ctx=h, q=p, q_stride=256, S=1, Tq=1, Hq=2, Hkv=1, D=128, kc=p, ks=p, vc=p, vs=p, P=2, page=4, lens=p, sm=None,
        bt=p, ld=2, dead=-1, scale=1.0, out=p, lse=None, stream=s), **kw}.values())
    assert att(S=0) == kv.OK and att(Tq=0) == kv.OK
    for code, kw in [(kv.ERR_INVALID_ARG, dict(q=None)), (kv.ERR_INVALID_ARG, dict(kc=None)), (kv.ERR_INVALID_ARG, dict(lens=None)),
                     (kv.ERR_INVALID_ARG, dict(sm=p)), (kv.ERR_INVALID_ARG, dict(bt=None)), (kv.ERR_INVALID_ARG, dict(scale=0.0)),
                     (kv.ERR_INVALID_ARG, dict(scale=float("nan"))), (kv.ERR_INVALID_ARG, dict(scale=float("inf"))),
                     (kv.ERR_SHAPE, dict(Hq=3, Hkv=2)), (kv.ERR_SHAPE, dict(S=-1)), (kv.ERR_SHAPE, dict(page=0)),
                     (kv.ERR_SHAPE, dict(q_stride=128)), (kv.ERR_UNSUPPORTED, dict(D=96)), (kv.ERR_UNSUPPORTED, dict(Tq=1025)),
                     (kv.ERR_UNSUPPORTED, dict(P=2 ** 30, page=4)), (kv.ERR_UNSUPPORTED, dict(ld=2 ** 30, page=4)),
                     (kv.ERR_ALIGN, dict(q=p + 2)), (kv.ERR_ALIGN, dict(q_stride=257)), (kv.ERR_ALIGN, dict(vs=p + 8)),
                     (kv.ERR_ALIGN, dict(out=p + 8))]:
        assert att(**kw) == code, kw
    pro = lambda **kw: kv.kvsel_prompt_attention(*{**dict(  # noqa: E731
        ctx=h, q=p, k=p, v=p, qs=256, ks=128, vs=128, cu=p, S=1, T=2, Hq=2, Hkv=1, D=128, scale=1.0, out=p, lse=None,
        stream=s), **kw}.values())
    assert pro(S=0) == kv.OK and pro(T=0) == kv.OK
    for code, kw in [(kv.ERR_INVALID_ARG, dict(k=None)), (kv.ERR_INVALID_ARG, dict(cu=None)), (kv.ERR_INVALID_ARG, dict(scale=-1.0)),
                     (kv.ERR_SHAPE, dict(Hq=3, Hkv=2)), (kv.ERR_SHAPE, dict(ks=64)), (kv.ERR_UNSUPPORTED, dict(D=256)),
                     (kv.ERR_UNSUPPORTED, dict(T=2 ** 25)), (kv.ERR_ALIGN, dict(v=p + 8)), (kv.ERR_ALIGN, dict(qs=260))]:
        assert pro(**kw) == code, kw
    sto = lambda **kw: kv.kvsel_kv4_store(*{**dict(  # noqa: E731
        ctx=h, k=p, v=p, dt=kv.BF16, ks=128, vs=128, T=1, Hkv=1, D=128, slots=p, kc=p, ksc=p, vc=p, vsc=p, P=1, page=4,
        stream=s), **kw}.values())
    assert sto(T=0) == kv.OK
    for code, kw in [(kv.ERR_INVALID_ARG, dict(dt=7)), (kv.ERR_INVALID_ARG, dict(slots=None)), (kv.ERR_INVALID_ARG, dict(vsc=None)),
                     (kv.ERR_SHAPE, dict(ks=64)), (kv.ERR_SHAPE, dict(page=0)), (kv.ERR_UNSUPPORTED, dict(D=80)),
                     (kv.ERR_ALIGN, dict(k=p + 2)), (kv.ERR_ALIGN, dict(vs=130)), (kv.ERR_ALIGN, dict(kc=p + 8))]:
        assert sto(**kw) == code, kw
    pln = lambda **kw: kv.kvsel_plan_slots(*{**dict(  # noqa: E731
        ctx=h, c=p, n=p, S=1, page=4, P=4, free=p, nf=1, bt=p, mb=2, cu=p, ns=p, np_=p, T=1, sm=None, ld=0, counts=p,
        stream=s), **kw}.values())
    for code, kw in [(kv.ERR_INVALID_ARG, dict(c=None)), (kv.ERR_INVALID_ARG, dict(cu=None)), (kv.ERR_INVALID_ARG, dict(ld=3)),
                     (kv.ERR_SHAPE, dict(page=0)), (kv.ERR_SHAPE, dict(T=-1)), (kv.ERR_UNSUPPORTED, dict(S=16385)),
                     (kv.ERR_UNSUPPORTED, dict(P=2 ** 30)), (kv.ERR_UNSUPPORTED, dict(mb=2 ** 30)),
                     (kv.ERR_UNSUPPORTED, dict(sm=p, ld=2 ** 31 - 1))]:
        assert pln(**kw) == code, kw
    torch.cuda.synchronize()
    assert not x.any()  # nothing was launched
    q = torch.zeros((2, 4, 64), dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        ctx.prompt_attention(q.half(), q, q, _i32([0, 2]), q)
    with pytest.raises(ValueError, match="back to back"):
        ctx.prompt_attention(q.transpose(0, 1), q, q, _i32([0, 2]), q)
    with pytest.raises(ValueError, match="k and v"):
        ctx.prompt_attention(q, q[:1], q, _i32([0, 2]), q)
    with pytest.raises(kv.KvselError, match="stride"):  # expanded tokens
        ctx.prompt_attention(q[:1].expand(2, 4, 64), q, q, _i32([0, 2]), torch.zeros_like(q))
    with pytest.raises(kv.KvselError, match="stride"):
        ctx.kv4_store(q[:1].expand(2, 4, 64), q, _i32([0, 1]), *_cache(1, 4, 4, 64))
    with pytest.raises(ValueError, match="evenly spaced"):
        ctx.kv4_attention(torch.zeros((2, 3, 2, 4, 64), dtype=BF, device="cuda")[:, :, 0][:, :2], *_cache(1, 4, 4, 64),
                          _i32([1, 1]), torch.zeros((2, 2, 4, 64), dtype=BF, device="cuda"),
                          block_table=_i32([[0], [0]]))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_serving_step_end_to_end(ctx):
    """Admission (plan, prompt attention, store), an IntentKV pruning of one session on the same slot map, two decode
    steps planned, stored and attended, on a side stream; every decode output against the formula on the stored rows."""
    page, Hq, Hkv, D, S = 16, 8, 2, 64, 3
    P, rows = 40, 8
    g = torch.Generator(device="cuda").manual_seed(21)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        prompts = [70, 1, 33]
        table = torch.full((S, rows), -1, dtype=I32, device="cuda")
        free = torch.randperm(P, generator=g, device="cuda").to(I32)
        cache = _cache(P, Hkv, page, D, 255)
        maps = torch.empty((S, rows * page), dtype=I32, device="cuda")
        counts = torch.empty(2, dtype=I32, device="cuda")
        cached = _i32([0, 0, 0])
        T = sum(prompts)

        def admit(new, T):
            cu, slots, pos = (torch.empty(n, dtype=I32, device="cuda") for n in (S + 1, T, T))
            ctx.plan_slots(cached, new, free, page, P, table, cu, slots, pos, counts, slot_map=maps)
            return cu, slots, pos

        cu, slots, pos = admit(_i32(prompts), T + 5)
        qkv = torch.randn((T + 5, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        out, lse = torch.zeros((T + 5, Hq, D), dtype=BF, device="cuda"), torch.zeros((T + 5, Hq), device="cuda")
        ctx.prompt_attention(q, k, v, cu, out, lse=lse)
        ctx.kv4_store(k, v, slots, *cache)
        ctx.check_device()
        _check_prompt(q, k, v, [0, 70, 71, 104], D ** -0.5, out, lse)
        taken = int(counts[1])
        assert counts.tolist() == [104, 5 + 1 + 3]

        # prune session 0 to 24 of its 70 tokens by rule scores on the stored keys, read back into a bf16 pool
        every = torch.arange(P * page, dtype=I32, device="cuda")
        kb, vb = (torch.empty((P * page, Hkv, D), dtype=BF, device="cuda") for _ in range(2))
        loaded = torch.where(torch.isin(every, slots[:T]), every, -1)
        ctx.kv4_load(*cache, loaded, kb, vb)
        M = torch.empty((1, Hq, D), device="cuda")
        ctx.memory_update(q[60:70].permute(1, 0, 2).contiguous()[None], 0.3, M, first_turn=True)
        rule, keep = torch.empty(70, device="cuda"), torch.empty(70, dtype=torch.uint8, device="cuda")
        sm0 = maps[0, :70].contiguous()
        ctx.rule_scores(kb[None], M, 1, Hq, Hkv, 70, D, 4, 60, 70, rule, slot_map=sm0, n_slots=P * page)
        n = ctx.topk_retain(rule, 4, 60, 70, 24, keep=keep)
        dead = P * page
        pruned = torch.empty_like(sm0)
        ctx.redirect_slots(sm0, keep, dead, pruned)
        assert n == 24

        lens = list(prompts)
        for step in range(2):
            cached = _i32(lens)
            free = free[taken:].contiguous()
            cu, slots, pos = admit(_i32([1, 1, 1]), 4)
            taken = int(counts[1])
            assert slots[3] == -1 and pos.tolist() == lens + [-1]
            maps[0, :70] = pruned
            x = torch.randn((4, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
            ctx.kv4_store(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots, *cache)
            lens = [n + 1 for n in lens]
            qd = x[:3, :Hq].unsqueeze(1)
            o, l = torch.empty((S, 1, Hq, D), dtype=BF, device="cuda"), torch.empty((S, 1, Hq), device="cuda")
            ctx.kv4_attention(qd, *cache, _i32(lens), o, slot_map=maps, dead_slot=dead, lse=l)
            ctx.check_device()
            sm = maps.cpu().numpy()
            live = (sm >= 0) & (sm != dead)
            assert live[0].sum() == 24 + step + 1
            _check_attention(o, l, _attention_reference(qd, cache, lens, np.where(live, sm, 0), live, D ** -0.5))
    torch.cuda.current_stream().wait_stream(side)


def test_decode_step_from_a_graph(ctx):
    """plan, store and attention captured once and replayed while the lengths move on; eager calls of other sizes on the
    same context in between change nothing."""
    page, Hq, Hkv, D, S, rows, P = 16, 4, 2, 128, 3, 12, 40
    g = torch.Generator(device="cuda").manual_seed(22)
    table = torch.randperm(P, generator=g, device="cuda").to(I32)[:S * rows].view(S, rows).contiguous()
    cache = _random_cache(g, P, Hkv, page, D)
    x = torch.randn((S, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
    cached, ones, free = _i32([40, 3, 150]), _i32([1, 1, 1]), _i32([39])
    cu, slots, pos, counts = (torch.empty(n, dtype=I32, device="cuda") for n in (S + 1, S, S, 2))
    lens = torch.empty_like(cached)
    out, lse = torch.empty((S, 1, Hq, D), dtype=BF, device="cuda"), torch.empty((S, 1, Hq), device="cuda")

    def step():
        ctx.plan_slots(cached, ones, free, page, P, table, cu, slots, pos, counts)
        ctx.kv4_store(x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], slots, *cache)
        torch.add(cached, ones, out=lens)
        ctx.kv4_attention(x[:, :Hq].unsqueeze(1), *cache, lens, out, block_table=table, lse=lse)

    start = [c.clone() for c in cache]
    step()  # warm-up on the capturing inputs
    torch.cuda.synchronize()
    for c, s in zip(cache, start):
        c.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    j = np.arange(rows * page)
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(BF))
        graph.replay()
        if i == 1:  # other sizes, eagerly, in between
            test_attention_is_deterministic(ctx)
        n = [40 + i + 1, 3 + i + 1, 150 + i + 1]
        tb = table.cpu().numpy()
        sl = tb[:, j // page] * page + j % page
        _check_attention(out, lse, _attention_reference(x[:, :Hq].unsqueeze(1), cache, n, sl, np.ones_like(sl, bool), D ** -0.5))
        cached += 1
    ctx.check_device()


def test_two_contexts_on_two_streams(ctx):
    """Decode and prompt attention of two contexts, on streams that run beside each other, as on one."""
    g = torch.Generator(device="cuda").manual_seed(24)
    Hq, Hkv, D, page, P = 8, 2, 128, 16, 256
    other = kv.Context(0)
    work = []
    for c, lens in ((ctx, [3000, 5]), (other, [900, 2500])):
        cache = _random_cache(g, P, Hkv, page, D)
        table = torch.randperm(P, generator=g, device="cuda").to(I32)[:2 * 120].view(2, 120) % P
        table = torch.cat([table, table], 1).contiguous()
        q = torch.randn((2, 1, Hq, D), generator=g, device="cuda").to(BF)
        x = torch.randn((700, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
        work.append((c, q, cache, _i32(lens), table, x, _i32([0, 300, 700]), torch.cuda.Stream()))

    def run(w, stream):
        c, q, cache, lens, table, x, cu, _ = w
        outs = []
        with torch.cuda.stream(stream):
            for _ in range(5):
                o, p = torch.empty_like(q), torch.empty((700, Hq, D), dtype=BF, device="cuda")
                c.kv4_attention(q, *cache, lens, o, block_table=table)
                c.prompt_attention(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cu, p)
                outs += [o, p]
        return outs

    want = [run(w, torch.cuda.current_stream()) for w in work]
    torch.cuda.synchronize()
    got = [run(w, w[-1]) for w in work]
    torch.cuda.synchronize()
    for c, a, b in zip((ctx, other), want, got):
        c.check_device()
        assert all(torch.equal(i, j) for i, j in zip(a, b))
    other.close()


def test_prompt_from_a_graph(ctx):
    """Captured once, replayed on other prompts of other lengths in the same buffers."""
    g = torch.Generator(device="cuda").manual_seed(33)
    T, Hq, Hkv, D = 900, 6, 2, 128
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda").to(BF)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cu = _i32([0, 300, 900])
    out, lse = torch.empty((T, Hq, D), dtype=BF, device="cuda"), torch.empty((T, Hq), device="cuda")
    ctx.prompt_attention(q, k, v, cu, out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ctx.prompt_attention(q, k, v, cu, out, lse=lse)
    for starts in ([0, 300, 900], [0, 1, 900], [0, 512, 640], [20, 20, 777]):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(BF))
        cu.copy_(_i32(starts))
        out.fill_(9)
        graph.replay()
        _check_prompt(q, k, v, starts, D ** -0.5, out, lse)
        assert (out[:starts[0]] == 9).all() and (out[starts[-1]:] == 9).all()
    ctx.check_device()
