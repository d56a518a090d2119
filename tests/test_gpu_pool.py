"""Attention over the bf16 page pools, attention mass and eviction by it, against plain 64-bit implementations (GB300)."""
import numpy as np
import pytest
import torch

import pool_reference as ref

pytestmark = pytest.mark.gpu

BF, I32, F32 = torch.bfloat16, torch.int32, torch.float32


@pytest.fixture(scope="module")
def ctx():
    import kv_cache_retention_gb300 as kv
    c = kv.Context(0)
    yield c
    c.close()


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=I32).cuda()


def _flagged(ctx, word):
    import kv_cache_retention_gb300 as kv
    with pytest.raises(kv.KvselError) as e:
        ctx.check_device()
    assert e.value.code == kv.ERR_DEVICE_CHECK and word in str(e.value), str(e.value)


class World:
    """Sessions over pools of random rows: packed queries, a block table or a slot map with dropped tokens."""

    def __init__(self, new, lens, Hq, Hkv, D, page, kind, seed=0, drop=0.4, extra=0, k_scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        S, rows = len(lens), -(-max(list(lens) + [1]) // page) + 1
        self.P, self.page, self.S, self.lens_host = S * rows + 1, page, S, list(lens)
        self.cu_host = [0] + [int(x) for x in np.cumsum(new)]
        T = self.cu_host[-1] + extra
        table = rng.permutation(self.P)[:S * rows].reshape(S, rows)
        j = np.arange(rows * page)
        slots = table[:, j // page] * page + j % page
        live = np.ones_like(slots, bool)
        self.dead = self.P * page
        self.args = dict(block_table=_i32(table))
        if kind == "map":  # some tokens at the dead slot, some at -1; what lies behind the length is not looked at
            u = rng.random(slots.shape)
            live = u > drop
            sm = np.where(u < drop / 2, self.dead, np.where(live, slots, -1))
            sm[j[None] >= np.array(lens)[:, None]] = 2 ** 31 - 1
            self.args = dict(slot_map=_i32(sm), dead_slot=self.dead)
        self.slots, self.live = torch.from_numpy(slots).cuda(), torch.from_numpy(live).cuda()
        self.q = torch.randn((T, Hq, D), generator=g, device="cuda").to(BF)
        self.k = (torch.randn((self.P, page, Hkv, D), generator=g, device="cuda") * k_scale).to(BF)
        self.v = torch.randn((self.P, page, Hkv, D), generator=g, device="cuda").to(BF)
        self.cu, self.lens, self.scale = _i32(self.cu_host), _i32(lens), D ** -0.5
        self.out = torch.full_like(self.q, 9)
        self.lse = torch.full((T, Hq), 9.0, device="cuda")

    def attend(self, ctx, **kw):
        ctx.pool_attention(*[kw.pop(n, getattr(self, n)) for n in ("q", "k", "v", "cu", "lens", "out")],
                           **{**dict(lse=self.lse, scale=self.scale), **self.args, **kw})

    def want(self):
        return ref.attend(self.q, self.k, self.v, self.cu_host, self.lens_host, self.slots, self.live, self.scale)

    def check(self, ctx):
        self.attend(ctx)
        ctx.check_device()
        ref.check_attend(self.out, self.lse, self.want())


SHAPES = [
    # new tokens, lengths, Hq, Hkv, D, page
    ([1], [1], 1, 1, 64, 1),
    ([1], [31], 4, 2, 64, 16),
    ([1, 1], [128, 33], 8, 1, 128, 16),
    ([1, 1, 1], [257, 129, 1], 10, 2, 128, 32),
    ([1, 1, 1, 1], [700, 5, 513, 1], 32, 8, 128, 16),
    ([4, 2], [2, 130], 8, 2, 128, 16),             # more new tokens than the session has: the first rows see nothing
    ([7, 0, 3], [100, 50, 61], 6, 2, 64, 7),       # a session without new tokens
    ([0, 1, 0], [0, 1, 40], 2, 1, 128, 16),
    ([3], [95], 16, 1, 128, 16),
    ([1], [200], 48, 1, 64, 3),                    # large groups of heads
    ([5], [77], 128, 1, 128, 16),
    ([2, 130], [400, 131], 100, 1, 64, 16),
    ([32, 33, 31, 64, 65], [32, 160, 159, 64, 321], 4, 1, 128, 16),
    ([128], [128], 2, 2, 128, 16),
    ([300, 1, 129], [300, 2000, 640], 4, 4, 64, 64),
    ([257], [1024], 5, 1, 128, 16),                # 25 tokens of five heads a tile
    ([333, 77, 1], [1999, 777, 1300], 14, 2, 64, 32),
    ([1], [5000], 5, 1, 128, 64),
    ([1], [9001], 16, 8, 128, 16),
    ([700], [701], 12, 12, 64, 8),
    ([1 + i % 3 for i in range(40)], [3 + 37 * i for i in range(40)], 8, 2, 64, 16),
    ([1] * 300, [1 + (i * i * 37) % 900 for i in range(299)] + [2500], 2, 1, 64, 16),
    ([1, 400, 1, 60, 1, 1, 9, 2, 150], [2100, 400, 1, 2100, 40, 7, 1000, 3, 2222], 8, 4, 128, 16),
    ([2, 1, 1], [767, 4000, 769], 160, 160, 64, 16),  # more kv heads than SMs
    ([900, 1, 500], [4900, 6000, 500], 32, 8, 128, 16),
    ([600], [600], 40, 8, 128, 16),
    # sessions of few tokens beside others, an odd number of kv heads, rows that just fill what the kernel for few takes
    ([1] * 20 + [100, 3], [40 + 133 * i for i in range(20)] + [777, 3000], 8, 2, 128, 16),
    ([1, 1, 1, 30], [2000, 300, 129, 500], 12, 3, 64, 16),
    ([2, 8, 9], [3000, 40, 900], 4, 1, 128, 16),
    ([8, 8, 7], [8, 300, 4000], 8, 2, 128, 16),
    ([1, 1], [900, 70], 64, 2, 128, 16),
    ([1, 2], [300, 200], 40, 1, 64, 16),
    ([1, 1, 0, 1], [3000, 20000, 5, 1], 6, 6, 64, 16),
    ([4] * 9, [500 * i + 4 for i in range(9)], 15, 5, 128, 32),
]


@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page", SHAPES)
@pytest.mark.parametrize("kind", ["table", "map"])
def test_attention_matches_reference(ctx, new, lens, Hq, Hkv, D, page, kind):
    World(new, lens, Hq, Hkv, D, page, kind, seed=len(lens) * 100 + Hq).check(ctx)


@pytest.mark.parametrize("kind", ["table", "map"])
def test_attention_of_few_live_tokens(ctx, kind):
    """A hundredth of long maps live, and sessions of which nothing is."""
    w = World([1, 40, 1, 3], [9000, 5000, 700, 128], 8, 2, 128, 16, "map", seed=3, drop=0.99)
    w.live[2] = w.live[3] = False
    w.args["slot_map"][2:] = w.dead
    w.check(ctx)
    assert torch.isinf(w.lse[41:]).all() and not w.out[41:].any()


def test_attention_never_reads_dropped_rows(ctx):
    """NaN rows in dropped slots, behind the lengths and in other sessions' pages change nothing."""
    w = World([2, 70], [200, 333], 8, 2, 128, 16, "map", seed=4)
    used = torch.zeros(w.P * w.page, dtype=torch.bool, device="cuda")
    for s in range(2):
        n = w.lens_host[s]
        used[w.slots[s, :n][w.live[s, :n]]] = True
    w.attend(ctx)
    clean = w.out.clone(), w.lse.clone()
    for pool in (w.k, w.v):
        pool[~used.view(w.P, w.page)] = float("nan")
    w.attend(ctx)
    ctx.check_device()
    assert torch.equal(w.out, clean[0]) and torch.equal(w.lse, clean[1])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,n", [(300, 300), (300, 4000), (40, 700), (3, 130)])
@pytest.mark.parametrize("Hkv", [2, 16])
def test_attention_future_nan_is_not_seen(ctx, D, new, n, Hkv):
    """NaN and infinite keys and values among the new tokens reach the rows at and behind them, and none before."""
    w = World([new], [n], 2 * Hkv, Hkv, D, 16, "table", seed=5)
    w.attend(ctx)
    clean = w.out.clone(), w.lse.clone()
    i, j = new // 2, 2 * new // 3
    at = lambda t: (w.slots[0, n - new + t] // 16, w.slots[0, n - new + t] % 16)  # noqa: E731
    for bad in (float("nan"), float("inf")):
        k, v = w.k.clone(), w.v.clone()
        k[(*at(i), 0, 5)] = float("nan")
        v[(*at(j), 1, 7)] = bad
        w.attend(ctx, k=k, v=v)
        ctx.check_device()
        assert torch.equal(w.out[:i, :2], clean[0][:i, :2]) and torch.isnan(w.out[i:, :2].float()).all()
        assert torch.equal(w.lse[:i, :2], clean[1][:i, :2]) and torch.isnan(w.lse[i:, :2]).all()
        assert torch.equal(w.out[:j, 2:4], clean[0][:j, 2:4]) and torch.equal(w.lse[:, 2:4], clean[1][:, 2:4])
        assert not torch.isfinite(w.out[j:, 2:4, 7].float()).any()
        others = [d for d in range(D) if d != 7]
        assert torch.equal(w.out[:, 2:4, others], clean[0][:, 2:4, others])
        assert torch.equal(w.out[:, 4:], clean[0][:, 4:])


def test_attention_values_behind_the_last_key_of_a_tile(ctx):
    """A NaN value that every row sees, and none: rows of a session that ends inside a tile."""
    w = World([1, 2], [129, 250], 4, 2, 64, 16, "table", seed=6)
    s, o = int(w.slots[1, 100] // 16), int(w.slots[1, 100] % 16)
    w.v[s, o, 0, 3] = float("inf")
    w.v[int(w.slots[1, 250] // 16), int(w.slots[1, 250] % 16), 1, 3] = float("nan")  # behind the length
    w.attend(ctx)
    ctx.check_device()
    assert torch.isinf(w.out[1:, :2, 3].float()).all()
    rest = torch.isfinite(w.out.float())
    rest[1:, :2, 3] = True
    assert rest.all()


def test_attention_rows_outside_sessions_stay(ctx):
    w = World([5, 200], [40, 1000], 4, 2, 128, 16, "map", seed=7, extra=31)
    w.check(ctx)
    assert (w.out[205:] == 9).all() and (w.lse[205:] == 9).all()
    cu = [3, 8, 208]                    # the first rows are nobody's either
    w.out.fill_(9), w.lse.fill_(9)
    w.attend(ctx, cu=_i32(cu))
    ctx.check_device()
    w.cu_host = cu
    ref.check_attend(w.out, w.lse, w.want())
    for t in (w.out, w.lse):
        assert (t[:3] == 9).all() and (t[208:] == 9).all()


@pytest.mark.parametrize("cu", [[0, 9], [5, -2 ** 31], [2 ** 31 - 1, 2 ** 31 - 1], [3, 2, 8], [-2 ** 31, 2 ** 31 - 1],
                                [0, 2 ** 31 - 1, 8], [600, 700], [0, 300, 100, 8]])
def test_attention_bad_sequences_are_flagged(ctx, cu):
    """Sequences outside the rows, or descending: flagged, and nothing outside the rows is written."""
    T, S = 8, len(cu) - 1
    w = World([8], [64], 2, 1, 64, 16, "table", seed=8, extra=1000)
    table = w.args["block_table"].expand(S, -1).contiguous()
    lens = _i32([64] * S)
    w.attend(ctx, q=w.q[:T], out=w.out[:T], lse=w.lse[:T], cu=_i32(cu), lens=lens, block_table=table)
    _flagged(ctx, "length out of range")
    assert (w.out[T:] == 9).all() and (w.lse[T:] == 9).all()
    score = torch.zeros((S, table.shape[1] * 16), device="cuda")
    ctx.attention_mass(w.q[:T], torch.zeros((T, 2), device="cuda"), w.k, _i32(cu), lens, score, block_table=table)
    _flagged(ctx, "length out of range")


def test_attention_bad_lengths_slots_and_pages(ctx):
    w = World([1, 3], [32, 32], 4, 1, 64, 16, "table", seed=9)
    table, slots, live = w.args["block_table"][:, :2].contiguous(), w.slots[:, :32], w.live[:, :32]
    score = torch.zeros((2, 32), device="cuda")
    for lens, cut in (([33, -1], [32, 0]), ([2 ** 31 - 1, -2 ** 31], [32, 0])):
        w.attend(ctx, lens=_i32(lens), block_table=table)
        _flagged(ctx, "length out of range")
        ref.check_attend(w.out, w.lse, ref.attend(w.q, w.k, w.v, w.cu_host, cut, slots, live, w.scale))
        ctx.attention_mass(w.q, w.lse, w.k, w.cu, _i32(lens), score, block_table=table, scale=w.scale)
        _flagged(ctx, "length out of range")
        ref.check_mass(score, ref.mass(w.q, w.lse, w.k, w.cu_host, cut, slots, live, w.scale, torch.zeros_like(score)))
    bad, live2 = table.clone(), live.clone()
    bad[0, 1], bad[1, 0] = w.P, -1
    live2[0, 16:], live2[1, :16] = False, False
    w.attend(ctx, block_table=bad)
    _flagged(ctx, "page out of range")
    ref.check_attend(w.out, w.lse, ref.attend(w.q, w.k, w.v, w.cu_host, w.lens_host, slots, live2, w.scale))
    ctx.attention_mass(w.q, w.lse, w.k, w.cu, w.lens, score, block_table=bad, scale=w.scale)
    _flagged(ctx, "page out of range")
    sm, live2 = slots.to(I32).contiguous(), live.clone()
    sm[0, 3], sm[1, 31], sm[1, 0] = w.P * 16, 2 ** 31 - 1, -2 ** 31
    live2[0, 3] = live2[1, 31] = live2[1, 0] = False
    w.attend(ctx, block_table=None, slot_map=sm)
    _flagged(ctx, "slot out of range")
    ref.check_attend(w.out, w.lse, ref.attend(w.q, w.k, w.v, w.cu_host, w.lens_host, slots, live2, w.scale))
    ctx.attention_mass(w.q, w.lse, w.k, w.cu, w.lens, score, slot_map=sm, scale=w.scale)
    _flagged(ctx, "slot out of range")
    ref.check_mass(score, ref.mass(w.q, w.lse, w.k, w.cu_host, w.lens_host, slots, live2, w.scale, torch.zeros_like(score)))


def test_attention_dead_slot_inside_the_pool(ctx):
    w = World([2], [150], 4, 2, 128, 16, "table", seed=10)
    sm = w.slots[:, :150].to(I32).contiguous()
    dead = int(sm[0, 40])
    live = torch.ones_like(sm, dtype=torch.bool)
    live[0, 40] = False
    w.attend(ctx, block_table=None, slot_map=sm, dead_slot=dead)
    ctx.check_device()
    ref.check_attend(w.out, w.lse, ref.attend(w.q, w.k, w.v, w.cu_host, w.lens_host, sm.long(), live, w.scale))


def test_attention_one_slot_for_many_tokens(ctx):
    """Tokens that share a slot (a prefix of two sessions; the same slot twice in one) count each by itself."""
    w = World([1, 33], [90, 90], 4, 2, 64, 16, "table", seed=11)
    sm = w.slots[:, :90].to(I32).contiguous()
    sm[1, :60] = sm[0, :60]
    sm[:, 7] = sm[0, 5]
    w.attend(ctx, block_table=None, slot_map=sm)
    ctx.check_device()
    ref.check_attend(w.out, w.lse, ref.attend(w.q, w.k, w.v, w.cu_host, w.lens_host, sm.long(), torch.ones_like(sm).bool(), w.scale))


def test_strided_rows_and_pools(ctx):
    """Queries out of a fused projection, pools that hold K and V of every slot side by side and several layers."""
    w = World([40, 1], [300, 777], 6, 2, 128, 16, "table", seed=12)
    w.attend(ctx)
    fused = torch.randn((41, 10, 128), device="cuda").to(BF)
    fused[:, :6] = w.q
    pools = torch.full((3, w.P, 16, 2, 2, 128), 7.0, device="cuda", dtype=BF)
    pools[1, :, :, 0], pools[1, :, :, 1] = w.k, w.v
    out, lse = torch.empty_like(w.out), torch.empty_like(w.lse)
    w.attend(ctx, q=fused[:, :6], k=pools[1, :, :, 0], v=pools[1, :, :, 1], out=out, lse=lse)
    only = torch.empty_like(out)
    w.attend(ctx, out=only, lse=None)
    score = [torch.empty((2, w.slots.shape[1]), device="cuda") for _ in range(2)]
    ctx.attention_mass(w.q, w.lse, w.k, w.cu, w.lens, score[0], **w.args)
    ctx.attention_mass(fused[:, :6], w.lse, pools[1, :, :, 0], w.cu, w.lens, score[1], **w.args)
    ctx.check_device()
    assert torch.equal(out, w.out) and torch.equal(lse, w.lse) and torch.equal(only, w.out) and torch.equal(*score)


def test_pools_past_32_bits(ctx):
    """Pools whose element offsets pass 2^32: rows at their end are read where they are."""
    D, Hkv, page = 128, 8, 32
    P = (1 << 32) // (Hkv * page * D) + 40
    w = World([1, 100], [700, 400], 16, Hkv, D, page, "table", seed=13)
    big = [torch.zeros((P, page, Hkv, D), dtype=BF, device="cuda") for _ in range(2)]
    for b, x in zip(big, (w.k, w.v)):
        b[P - w.P:] = x
    w.attend(ctx)
    out, lse = torch.empty_like(w.out), torch.empty_like(w.lse)
    far = dict(block_table=w.args["block_table"] + (P - w.P))
    w.attend(ctx, k=big[0], v=big[1], out=out, lse=lse, **far)
    score = [torch.empty((2, w.slots.shape[1]), device="cuda") for _ in range(2)]
    ctx.attention_mass(w.q, w.lse, w.k, w.cu, w.lens, score[0], **w.args)
    ctx.attention_mass(w.q, w.lse, big[0], w.cu, w.lens, score[1], **far)
    ctx.check_device()
    assert torch.equal(out, w.out) and torch.equal(lse, w.lse) and torch.equal(*score)


@pytest.mark.parametrize("qs,scale", [(1.0, 20.0), (60.0, 1.0), (1e-20, 1.0), (2.0 ** 50, 2.0 ** -50)])
@pytest.mark.parametrize("new", [1, 500])
def test_attention_extreme_logits(ctx, qs, scale, new):
    """Logits of thousands (one weight near 1), rising along the session, and of nothing (the mean)."""
    w = World([new], [700], 4, 2, 64, 16, "table", seed=14)
    w.q = (w.q.float() * qs).to(BF)
    up = torch.linspace(0.1, 3, 700, device="cuda")
    flat = w.k.flatten(0, 1)
    flat[w.slots[0, :700]] = (flat[w.slots[0, :700]].float() * up[:, None, None]).to(BF)
    w.scale = scale
    w.check(ctx)


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("new", [1, 150])
def test_attention_minus_infinite_logits(ctx, first, new):
    """Keys whose logits are -inf for every row, at the session's start or its end: as if they were dropped."""
    n, page = 900, 16
    w = World([new], [n], 4, 2, 64, page, "table", seed=15)
    w.q[..., 0] = 1
    hidden = w.slots[0, :300] if first else w.slots[0, 700:n]
    w.k.flatten(0, 1)[hidden] = 0
    w.k.flatten(0, 1)[hidden, :, 0] = -float("inf")
    w.attend(ctx)
    ctx.check_device()
    live = torch.ones_like(w.live)
    live[0, :300 if first else 0] = False
    live[0, n if first else 700:] = False
    clean = w.k.clone()
    clean.flatten(0, 1)[hidden] = 0
    ref.check_attend(w.out, w.lse, ref.attend(w.q, clean, w.v, w.cu_host, w.lens_host, w.slots, live, w.scale))


def test_attention_is_deterministic_and_captured(ctx):
    """Two captured calls of one context, replayed in turn with eager calls between them, bit for bit."""
    cases = []
    for new, lens, Hq, Hkv, D in (([1, 1], [4000, 3000], 8, 2, 128), ([300, 1, 40], [2500, 2000, 1111], 6, 1, 64)):
        w = World(new, lens, Hq, Hkv, D, 16, "map", seed=Hq)
        score = torch.empty((w.S, w.slots.shape[1]), device="cuda")

        def call(w=w, score=score):
            w.attend(ctx)
            ctx.attention_mass(w.q, w.lse, w.k, w.cu, w.lens, score, scale=w.scale, **w.args)
        call()
        torch.cuda.synchronize()
        want = w.out.clone(), w.lse.clone(), score.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        cases.append((graph, call, w, score, want))
    for i in range(6):
        for n, (graph, call, w, score, want) in enumerate(cases):
            for t in (w.out, w.lse, score):
                t.fill_(7)
            graph.replay() if (i + n) % 3 else call()
            assert all(torch.equal(a, b) for a, b in zip((w.out, w.lse, score), want))
    ctx.check_device()


def test_calls_on_other_streams(ctx):
    """Two contexts on two streams at once give what each gives alone."""
    import kv_cache_retention_gb300 as kv
    other = kv.Context(0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    worlds = [World([200, 1], [3000, 5000], 8, 2, 128, 16, "map", seed=20 + i) for i in range(2)]
    scores = [torch.empty((2, w.slots.shape[1]), device="cuda") for w in worlds]
    maps = [w.args["slot_map"].clone() for w in worlds]

    def run(i, c, stream):
        w = worlds[i]
        w.attend(c, stream=stream)
        c.attention_mass(w.q, w.lse, w.k, w.cu, w.lens, scores[i], scale=w.scale, stream=stream, **w.args)
        c.evict_slots(scores[i], w.lens, _i32([900, 1000]), w.args["slot_map"], w.dead, maps[i], stream=stream)
    torch.cuda.synchronize()
    for i in range(2):
        run(i, ctx, None)
    torch.cuda.synchronize()
    want = [(w.out.clone(), w.lse.clone(), s.clone(), m.clone()) for w, s, m in zip(worlds, scores, maps)]
    budgets = torch.cuda.current_stream()
    for st in streams:
        st.wait_stream(budgets)
    for _ in range(5):
        for i, c in enumerate((ctx, other)):
            with torch.cuda.stream(streams[i]):
                run(i, c, streams[i])
    torch.cuda.synchronize()
    for i, (w, s, m) in enumerate(zip(worlds, scores, maps)):
        assert all(torch.equal(a, b) for a, b in zip((w.out, w.lse, s, m), want[i]))
    ctx.check_device(), other.check_device()
    other.close()


def test_no_sessions_and_no_tokens(ctx):
    w = World([1], [8], 2, 1, 64, 16, "table", seed=1)
    ctx.pool_attention(w.q[:0], w.k, w.v, _i32([0, 0]), w.lens, w.out[:0], lse=w.lse[:0], **w.args)
    assert (w.out == 9).all() and (w.lse == 9).all()
    none = torch.empty((0, 2), dtype=I32, device="cuda")
    ctx.pool_attention(w.q, w.k, w.v, _i32([0]), _i32([]), w.out, block_table=none)
    assert (w.out == 9).all()
    score, before = torch.full((1, 32), 5.0, device="cuda"), torch.arange(32.0, device="cuda")[None]
    ctx.attention_mass(w.q[:0], w.lse[:0], w.k, _i32([0, 0]), w.lens, score, score_in=before, **w.args)
    assert torch.equal(score, before)
    ctx.attention_mass(w.q[:0], w.lse[:0], w.k, _i32([0, 0]), w.lens, score, **w.args)
    assert not score.any()
    ctx.evict_slots(score[:0], _i32([]), _i32([]), none, 9, none)
    empty = torch.empty((1, 0), dtype=I32, device="cuda")
    freed, n = torch.full((1, 3), 7, dtype=I32, device="cuda"), torch.full((1,), 7, dtype=I32, device="cuda")
    ctx.evict_slots(torch.empty((1, 0), device="cuda"), _i32([0]), _i32([0]), empty, 9, empty, freed=freed, n_freed=n)
    ctx.check_device()
    assert freed.tolist() == [[-1] * 3] and n.tolist() == [0]


# ---------------------------------------------------------------------------
# attention_mass
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("new,lens,Hq,Hkv,D,page", SHAPES)
@pytest.mark.parametrize("kind", ["table", "map"])
def test_mass_matches_reference(ctx, new, lens, Hq, Hkv, D, page, kind):
    w = World(new, lens, Hq, Hkv, D, page, kind, seed=len(lens) * 100 + Hq)
    lse = torch.nan_to_num(w.want()[1], nan=9.0, neginf=-float("inf")).to(F32)
    g = torch.Generator(device="cuda").manual_seed(1)
    n = w.slots.shape[1]
    before = torch.rand((w.S, n + 5), generator=g, device="cuda")
    score = torch.full_like(before, 7)
    ctx.attention_mass(w.q, lse, w.k, w.cu, w.lens, score, score_in=before, scale=w.scale, **w.args)
    zero = torch.full_like(before, 7)
    ctx.attention_mass(w.q, lse, w.k, w.cu, w.lens, zero, scale=w.scale, **w.args)
    same = before.clone()
    ctx.attention_mass(w.q, lse, w.k, w.cu, w.lens, same, score_in=same, scale=w.scale, **w.args)
    ctx.check_device()
    args = (w.q, lse, w.k, w.cu_host, w.lens_host, w.slots, w.live, w.scale)
    ref.check_mass(score[:, :n], ref.mass(*args, before[:, :n]))
    ref.check_mass(zero[:, :n], ref.mass(*args, torch.zeros_like(before[:, :n])))
    assert torch.equal(same[:, :n], score[:, :n]) and torch.equal(same[:, n:], before[:, n:])
    assert (score[:, n:] == 7).all() and (zero[:, n:] == 7).all()
    unseen = ~w.live | (torch.arange(n, device="cuda")[None] >= w.lens[:, None])
    assert torch.equal(score[:, :n][unseen], before[:, :n][unseen])


def test_mass_of_all_rows_is_one_each(ctx):
    """The weights of a row sum to one: a session's scores add up to its rows, whatever their order in memory."""
    w = World([150, 1, 64], [4000, 333, 64], 12, 4, 128, 16, "map", seed=21)
    w.attend(ctx)
    score = torch.empty((3, w.slots.shape[1]), device="cuda")
    ctx.attention_mass(w.q, w.lse, w.k, w.cu, w.lens, score, scale=w.scale, **w.args)
    ctx.check_device()
    rows = torch.stack([(~torch.isinf(w.lse[a:b])).sum() for a, b in zip(w.cu_host[:-1], w.cu_host[1:])])
    # each weight's exponent is off by (D + 2) 2^-23 of its logit's absolute sum, below 100 here, in both calls
    assert ((score.double().sum(1) - rows).abs() <= rows * (2 * 130 * 2.0 ** -23 * 100)).all()


def test_mass_nan_keys_reach_their_own_token_alone(ctx):
    w = World([40], [500], 4, 2, 128, 16, "map", seed=22)
    lse = torch.nan_to_num(w.want()[1], neginf=-float("inf")).to(F32)
    score = [torch.empty((1, w.slots.shape[1]), device="cuda") for _ in range(2)]
    ctx.attention_mass(w.q, lse, w.k, w.cu, w.lens, score[0], scale=w.scale, **w.args)
    used = torch.zeros(w.P * 16, dtype=torch.bool, device="cuda")
    used[w.slots[0, :500][w.live[0, :500]]] = True
    w.k[~used.view(w.P, 16)] = float("nan")
    hit = int(torch.nonzero(w.live[0, :460]).flatten()[-1])
    late = int(torch.nonzero(w.live[0, :490]).flatten()[-1])  # among the new tokens
    for j in (hit, late):
        w.k[w.slots[0, j] // 16, w.slots[0, j] % 16, 1, 3] = float("nan")
    ctx.attention_mass(w.q, lse, w.k, w.cu, w.lens, score[1], scale=w.scale, **w.args)
    ctx.check_device()
    assert torch.isnan(score[1][0, [hit, late]]).all()
    score[1][0, [hit, late]] = score[0][0, [hit, late]]
    assert torch.equal(*score)


def test_mass_rows_that_see_nothing_or_belong_to_nobody(ctx):
    """Queries behind the sessions and rows with lse = -inf add nothing, whatever they hold."""
    w = World([3, 5], [200, 3], 4, 2, 64, 16, "table", seed=23, extra=40)
    lse = torch.nan_to_num(w.want()[1], nan=0.0, neginf=-float("inf")).to(F32)
    assert torch.isinf(lse[3:5]).all()
    want = ref.mass(w.q, lse, w.k, w.cu_host, w.lens_host, w.slots, w.live, w.scale, torch.zeros((2, w.slots.shape[1]), device="cuda"))
    w.q[8:], w.q[3:5] = float("nan"), float("nan")
    lse[8:] = float("nan")
    score = torch.empty((2, w.slots.shape[1]), device="cuda")
    ctx.attention_mass(w.q, lse, w.k, w.cu, w.lens, score, scale=w.scale, **w.args)
    ctx.check_device()
    ref.check_mass(score, want)


# ---------------------------------------------------------------------------
# evict_slots
# ---------------------------------------------------------------------------

def _evict_case(S, ld, seed, live=0.7, ties=0.3, low=0):
    rng = np.random.default_rng(seed)
    lens = rng.integers(low, ld + 1, S)
    slots = rng.permutation(S * ld).reshape(S, ld).astype(np.int64)
    dead = S * ld
    u = rng.random((S, ld))
    slots = np.where(u < live, slots, np.where(u < live + (1 - live) / 2, dead, -1 - (u * 50).astype(int)))
    score = rng.standard_normal((S, ld + 3)).astype(np.float32)
    score = np.where(rng.random(score.shape) < ties, np.round(score), score)
    score = np.where(rng.random(score.shape) < 0.02, np.nan, score)
    score = np.where(rng.random(score.shape) < 0.02, np.inf, score)
    score = np.where(rng.random(score.shape) < 0.02, -np.inf, score)
    score = np.where(rng.random(score.shape) < 0.02, -0.0, score).astype(np.float32)
    budget = np.array([rng.integers(0, max(1, int(n * live)) + 1) for n in lens])
    return rng, lens, slots, dead, score, budget


def _evict(ctx, score, lens, budget, slots, dead, sink, recent, room=None, alias=False):
    S, ld = slots.shape
    maps = _i32(slots)
    out = maps if alias else torch.full_like(maps, 12345)
    freed = None if room is None else torch.full((S, room), 12345, dtype=I32, device="cuda")
    n = torch.full((S,), 12345, dtype=I32, device="cuda")
    ctx.evict_slots(torch.from_numpy(score).cuda(), _i32(lens), _i32(budget), maps, dead, out, n_sink=sink, n_recent=recent,
                    freed=freed, n_freed=n)
    want, want_freed, want_n = ref.evict(score, lens, budget, slots, dead, sink, recent, room)
    assert np.array_equal(out.cpu().numpy(), want) and n.tolist() == want_n
    if room is not None:
        assert freed.tolist() == [f + [-1] * (room - len(f)) for f in want_freed]
    if not alias:
        assert torch.equal(maps, _i32(slots))


@pytest.mark.parametrize("S,ld", [(1, 1), (1, 31), (3, 33), (2, 1000), (5, 1025), (1, 5000), (40, 700), (300, 90), (1, 20001),
                                  (20, 9000), (160, 2049)])
@pytest.mark.parametrize("sink,recent,room", [(0, 0, None), (4, 32, 1), (3, 7, 64), (0, 100, 5000)])
def test_evict_matches_reference(ctx, S, ld, sink, recent, room):
    _, lens, slots, dead, score, budget = _evict_case(S, ld, S + ld)
    _evict(ctx, score, lens, budget, slots, dead, sink, recent, room, alias=room == 64)
    ctx.check_device()


@pytest.mark.parametrize("S,ld", [(1, 300000), (2, 270001), (160, 33000)])
def test_evict_rows_longer_than_shared_memory(ctx, S, ld):
    """More positions than the blocks of a session hold: scores and slots are read again for each pass."""
    _, lens, slots, dead, score, budget = _evict_case(S, ld, 5, low=ld - 5)
    _evict(ctx, score, lens, budget, slots, dead, 4, 32, 999)
    ctx.check_device()


@pytest.mark.parametrize("value", [0.0, float("nan"), float("inf"), -1.0])
def test_evict_equal_scores(ctx, value):
    """All scores alike: the latest positions that may leave do."""
    S, ld = 3, 4097
    slots = np.arange(S * ld).reshape(S, ld)
    score = np.full((S, ld), value, np.float32)
    _evict(ctx, score, [ld, 4000, 1], [ld - 1, 100, 0], slots, S * ld, 2, 5, 2000)
    _evict(ctx, score, [ld, 4000, 1], [ld - 1, 100, 0], slots, S * ld, 0, 0, 4096)


def test_evict_budgets_and_protected_positions(ctx):
    S, ld = 6, 500
    slots = np.arange(S * ld).reshape(S, ld)
    score = np.random.default_rng(3).random((S, ld)).astype(np.float32)
    lens, budget = [500, 500, 500, 500, 20, 0], [0, -5, 2 ** 31 - 1, 500, 3, 0]
    for sink, recent in ((0, 0), (100, 350), (300, 300), (2 ** 31 - 1, 0), (0, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1)):
        _evict(ctx, score, lens, budget, slots, S * ld, sink, recent, 500)
    _evict(ctx, score, lens, [-2 ** 31] * S, slots, S * ld, 1, 1)
    ctx.check_device()


def test_evict_lengths_out_of_range(ctx):
    slots = np.arange(3 * 64).reshape(3, 64)
    score = np.random.default_rng(4).random((3, 64)).astype(np.float32)
    _evict(ctx, score, [65, -1, 2 ** 31 - 1], [10, 10, 10], slots, 192, 0, 0, 64)
    _flagged(ctx, "length out of range")


def test_evict_captured(ctx):
    rng, lens, slots, dead, score, budget = _evict_case(7, 3000, 8)
    sc, maps, n = torch.from_numpy(score).cuda(), _i32(slots), torch.zeros(7, dtype=I32, device="cuda")
    out, le, bu = torch.empty_like(maps), _i32(lens), _i32(budget)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ctx.evict_slots(sc, le, bu, maps, dead, out, n_freed=n)
    for seed in (9, 10):
        _, lens, slots, dead, score, budget = _evict_case(7, 3000, seed)
        for t, x in ((sc, score), (maps, slots), (le, lens), (bu, budget)):
            t.copy_(torch.from_numpy(np.asarray(x)).to(t.dtype))
        graph.replay()
        want, _, counts = ref.evict(score, lens, budget, slots, dead, 0, 0)
        assert np.array_equal(out.cpu().numpy(), want) and n.tolist() == counts
    ctx.check_device()


# ---------------------------------------------------------------------------
# a run of them together
# ---------------------------------------------------------------------------

def test_prompts_then_decode_at_a_budget(ctx):
    """Prompts in chunks, then decode steps: plan, store, attend, weigh, evict; freed slots take the next tokens, so that
    no session's live tokens pass its budget and the pool does not grow."""
    S, Hq, Hkv, D, page, ld = 3, 8, 2, 64, 16, 512
    budget, sink, recent = [96, 120, 64], 4, 16
    prompts, chunk, steps = [200, 77, 130], 70, 12
    P = 64
    g = torch.Generator(device="cuda").manual_seed(30)
    k_pool, v_pool = (torch.zeros((P, page, Hkv, D), dtype=BF, device="cuda") for _ in range(2))
    dead = P * page
    maps = torch.full((S, ld), dead, dtype=I32, device="cuda")
    score, b = torch.zeros((S, ld), device="cuda"), _i32(budget)
    ref_score = torch.zeros((S, ld), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(ref_score)
    table = torch.full((S, ld // page), -1, dtype=I32, device="cuda")
    free, taken = torch.arange(P, dtype=I32, device="cuda"), 0
    done = [0] * S
    freed = torch.full((S, 64), -1, dtype=I32, device="cuda")
    n_freed = torch.zeros(S, dtype=I32, device="cuda")

    def step(new, slots, pos):
        nonlocal ref_score, tol
        T, cu = sum(new), [0] + [int(x) for x in np.cumsum(new)]
        sess = torch.repeat_interleave(torch.arange(S, device="cuda"), torch.tensor(new, device="cuda"))
        q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv))
        maps[sess, pos.long()] = slots
        k_pool.flatten(0, 1)[slots.long()], v_pool.flatten(0, 1)[slots.long()] = k, v
        lens_host = [d + n for d, n in zip(done, new)]
        lens, out, lse = _i32(lens_host), torch.empty_like(q), torch.empty((T, Hq), device="cuda")
        live = (maps >= 0) & (maps != dead)
        ctx.pool_attention(q, k_pool, v_pool, _i32(cu), lens, out, slot_map=maps, dead_slot=dead, lse=lse)
        ref.check_attend(out, lse, ref.attend(q, k_pool, v_pool, cu, lens_host, maps.long(), live, D ** -0.5))
        ctx.attention_mass(q, lse, k_pool, _i32(cu), lens, score, slot_map=maps, dead_slot=dead, score_in=score)
        ref_score, t = ref.mass(q, lse, k_pool, cu, lens_host, maps.long(), live, D ** -0.5, ref_score)
        tol = tol + t
        ref.check_mass(score, (ref_score, tol))
        before = maps.cpu().numpy()
        ctx.evict_slots(score, lens, b, maps, dead, maps, n_sink=sink, n_recent=recent, freed=freed, n_freed=n_freed)
        want, lists, counts = ref.evict(score.cpu().numpy(), lens_host, budget, before, dead, sink, recent, 64)
        assert np.array_equal(maps.cpu().numpy(), want) and n_freed.tolist() == counts
        assert [row[:c] for row, c in zip(freed.tolist(), counts)] == lists
        done[:] = lens_host

    while any(d < p for d, p in zip(done, prompts)):   # chunks of the prompts, slots from fresh pages
        new = [min(chunk, p - d) for d, p in zip(done, prompts)]
        T = sum(new)
        cu, slots, pos, counts = (torch.empty(n, dtype=I32, device="cuda") for n in (S + 1, T, T, 2))
        ctx.plan_slots(_i32(done), _i32(new), free[taken:].contiguous(), page, P, table, cu, slots, pos, counts)
        taken += int(counts[1])
        step(new, slots, pos)
    while any(int(((maps[s] >= 0) & (maps[s] != dead)).sum()) > budget[s] for s in range(S)):  # at most 64 leave a call
        ctx.evict_slots(score, _i32(done), b, maps, dead, maps, n_sink=sink, n_recent=recent, freed=freed, n_freed=n_freed)
    for _ in range(steps):                              # each new token takes a slot that its session gave up
        spare = torch.stack([freed[s, 0] if int(n_freed[s]) else free[taken + s] * page for s in range(S)])
        step([1] * S, spare, _i32(done))
    ctx.check_device()
    assert [int(((maps[s] >= 0) & (maps[s] != dead)).sum()) for s in range(S)] == [min(x, d) for x, d in zip(budget, done)]


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def test_refusals(ctx):
    import kv_cache_retention_gb300 as kv
    h, s = ctx.handle, torch.cuda.current_stream().cuda_stream
    x = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    p = x.data_ptr()
    att = lambda **kw: kv.kvsel_pool_attention(*{**dict(  # noqa: E731
        ctx=h, q=p, qs=256, cu=p, S=1, T=1, Hq=2, Hkv=1, D=128, k=p, v=p, ks=128, vs=128, P=2, page=4, lens=p, sm=None, bt=p,
        ld=1, dead=-1, scale=0.1, out=p, lse=None, stream=s), **kw}.values())
    mass = lambda **kw: kv.kvsel_attention_mass(*{**dict(  # noqa: E731
        ctx=h, q=p, qs=256, lse=p, cu=p, S=1, T=1, Hq=2, Hkv=1, D=128, k=p, ks=128, P=2, page=4, lens=p, sm=None, bt=p, ld=1,
        dead=-1, scale=0.1, before=None, score=p, score_ld=4, stream=s), **kw}.values())
    for call in (att, mass):
        for code, kws in {
            kv.ERR_SHAPE: [dict(S=-1), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=3, Hkv=2), dict(page=0), dict(ld=-1),
                           dict(P=-1), dict(T=2, qs=128), dict(ks=64)],
            kv.ERR_UNSUPPORTED: [dict(D=32), dict(D=256), dict(D=96), dict(Hq=129), dict(S=65536), dict(T=(1 << 24) + 1),
                                 dict(P=1 << 29), dict(ld=1 << 30), dict(Hq=65536, Hkv=65536, qs=65536 * 128)],
            kv.ERR_INVALID_ARG: [dict(bt=None), dict(sm=p), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                                 dict(scale=float("inf")), dict(q=None), dict(k=None), dict(cu=None), dict(lens=None)],
            kv.ERR_ALIGN: [dict(q=p + 8), dict(k=p + 2), dict(qs=257), dict(ks=132)],
        }.items():
            for kw in kws:
                assert call(**kw) == code, (kw, kv.kvsel_last_error_string(h))
                assert kv.kvsel_last_error_string(h)
    for kw, code in ((dict(v=None), kv.ERR_INVALID_ARG), (dict(out=None), kv.ERR_INVALID_ARG), (dict(out=p + 4), kv.ERR_ALIGN),
                     (dict(v=p + 8), kv.ERR_ALIGN), (dict(vs=129), kv.ERR_ALIGN), (dict(vs=8), kv.ERR_SHAPE)):
        assert att(**kw) == code, kw
    for kw, code in ((dict(lse=None), kv.ERR_INVALID_ARG), (dict(score=None), kv.ERR_INVALID_ARG),
                     (dict(S=2, score_ld=3), kv.ERR_SHAPE)):
        assert mass(**kw) == code, kw
    ev = lambda **kw: kv.kvsel_evict_slots(*{**dict(  # noqa: E731
        ctx=h, score=p, score_ld=8, lens=p, budget=p, S=1, sm=p, ld=8, dead=99, sink=0, recent=0, out=p, freed=p, ldf=4, nf=p,
        stream=s), **kw}.values())
    for kw, code in ((dict(S=-1), kv.ERR_SHAPE), (dict(ld=-1), kv.ERR_SHAPE), (dict(sink=-1), kv.ERR_SHAPE),
                     (dict(recent=-1), kv.ERR_SHAPE), (dict(ldf=-1), kv.ERR_SHAPE), (dict(freed=None), kv.ERR_SHAPE),
                     (dict(S=2, score_ld=7), kv.ERR_SHAPE), (dict(S=65536), kv.ERR_UNSUPPORTED),
                     (dict(ld=2 ** 31 - 1), kv.ERR_UNSUPPORTED), (dict(score=None), kv.ERR_INVALID_ARG),
                     (dict(lens=None), kv.ERR_INVALID_ARG), (dict(budget=None), kv.ERR_INVALID_ARG),
                     (dict(sm=None), kv.ERR_INVALID_ARG), (dict(out=None), kv.ERR_INVALID_ARG)):
        assert ev(**kw) == code, kw
    torch.cuda.synchronize()
    assert not x.any()


def test_binding_refusals(ctx):
    w = World([2], [40], 4, 2, 64, 16, "map", seed=1)
    ok = dict(w.args)
    bad = [dict(out=w.out[:1]), dict(lse=w.lse[:1]), dict(v=w.v[:, :8]), dict(k=w.k[..., :32]), dict(q=w.q.float()),
           dict(q=w.q.cpu()), dict(cu=w.cu[:1]), dict(lens=w.lens.long()), dict(slot_map=ok["slot_map"][0]),
           dict(slot_map=None), dict(block_table=ok["slot_map"]), dict(k=w.k.float()), dict(out=w.out.transpose(0, 1)),
           dict(v=w.v.transpose(1, 2)), dict(q=w.q.transpose(1, 2))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            w.attend(ctx, **kw)
    score = torch.zeros((1, w.slots.shape[1]), device="cuda")
    for kw in (dict(score=score[:, :-1]), dict(score=score[0]), dict(score=score.double()), dict(lse=w.lse[:1]),
               dict(score_in=score[:, :3]), dict(score_in=score.cpu())):
        a = {**dict(score=score, lse=w.lse, score_in=None), **kw}
        with pytest.raises((ValueError, TypeError)):
            ctx.attention_mass(w.q, a["lse"], w.k, w.cu, w.lens, a["score"], score_in=a["score_in"], **ok)
    sm = ok["slot_map"]
    for kw in (dict(out=sm[:, :-1]), dict(budget=w.cu), dict(freed=sm[:, :0]), dict(freed=sm[0]), dict(n_freed=w.cu),
               dict(score=score[:, :5]), dict(score=score.to(BF)), dict(out=sm.long())):
        a = {**dict(score=score, budget=w.lens, out=sm, freed=None, n_freed=None), **kw}
        with pytest.raises((ValueError, TypeError)):
            ctx.evict_slots(a["score"], w.lens, a["budget"], sm, w.dead, a["out"], freed=a["freed"], n_freed=a["n_freed"])
    torch.cuda.synchronize()
