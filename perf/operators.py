"""The serving operators around the retention path, each in its plain form and as the library's call.

  plan    plan_slots: block tables, slots and positions of a step's new tokens, slot maps of the sessions
  store   kv4_store + kv4_load: rows written to the 4-bit paged cache and read back from it
  decode  kv4_attention: attention of one or a few query rows per session over the 4-bit cache
  prompt  prompt_attention: causal attention over packed prompts with grouped heads

``run`` computes a case's operator in elementary torch operations while ``own`` is false, and with the calls of
kv_cache_retention_gb300 while it is true.

The 4-bit cache.  A row of D values is cut into groups of 16.  A group is stored as 16 four-bit E2M1 codes (sign, then
the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) and one scale byte, which holds bits 14..7 of the scale's fp16 pattern
(5 exponent and 3 mantissa bits): the smallest such scale s with max|x| <= 6 s.  Codes are the nearest to x / s, ties
to the even code.  A group that holds a NaN or a value above 61440 is stored as NaN (scale byte 255, codes 0).  Byte
i of a group's 8 holds the codes of its values 2i (low four bits) and 2i + 1.  Caches are [P][Hkv][page][...].
"""
import math

import numpy as np
import torch

own = False

DEVICE = "cuda"
GROUP = 16
TOP_BYTE = 226                    # the largest scale in use: 10240, so that 6 * scale stays below fp16's largest value
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# borders between neighbouring magnitudes, and whether a tie goes up (to the even code)
BORDERS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False))


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of a serving batch: 36 sessions, one new token each, and the sessions' slot maps
        dict(name="plan decode 36", op="plan", S=36, low=1024, high=8192, new_low=1, new_high=1, page=16, maps=True, pad=0),
        # admission of 64 sessions with long histories: prompts of up to 2048 new tokens, all slot maps
        dict(name="plan admit 64 long", op="plan", S=64, low=0, high=92160, new_low=0, new_high=2048, page=16, maps=True,
             pad=1024),
        # the rows of one decode step of 36 sessions (one layer)
        dict(name="store decode 36", op="store", T=36, Hkv=8, D=128, page=16, dtype="bf16", fused=True, skip=0.0),
        # a prompt of 32768 tokens written to the cache (one layer)
        dict(name="store prompt 32768", op="store", T=32768, Hkv=8, D=128, page=16, dtype="bf16", fused=True, skip=0.0),
        # the smallest call: one session of a small model
        dict(name="decode tiny", op="decode", S=1, Tq=1, Hq=4, Hkv=2, D=64, low=2048, high=2048, page=16, maps=False,
             live=1.0),
        # 36 sessions after pruning to a quarter: slot maps of 32768 positions whose dropped tokens point at the dead slot
        dict(name="decode pruned 36", op="decode", S=36, Tq=1, Hq=32, Hkv=8, D=128, low=20000, high=32768, page=16,
             maps=True, live=0.25),
        # one long session, groups of five heads, block tables with pages of 32
        dict(name="decode long 92160", op="decode", S=1, Tq=1, Hq=40, Hkv=8, D=128, low=92160, high=92160, page=32,
             maps=False, live=1.0),
        # drafted tokens checked four at a time: 16 sessions of uneven length
        dict(name="decode drafts 16", op="decode", S=16, Tq=4, Hq=32, Hkv=8, D=128, low=301, high=32768, page=16, maps=False,
             live=1.0),
        # a short prompt of a small model
        dict(name="prompt tiny", op="prompt", S=1, T=512, low=512, Hq=4, Hkv=2, D=64, fused=True),
        # one prompt of ordinary length
        dict(name="prompt 4096", op="prompt", S=1, T=4096, low=4096, Hq=32, Hkv=8, D=128, fused=True),
        # a packed batch: 9 prompts of uneven length, the shortest a single token
        dict(name="prompt packed 9", op="prompt", S=9, T=14700, low=1, Hq=32, Hkv=8, D=128, fused=True),
        # one long prompt, groups of five heads
        dict(name="prompt 16384", op="prompt", S=1, T=16384, low=16384, Hq=40, Hkv=8, D=128, fused=False),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "decode", "prompt"])
    if op == "plan":
        S = _log(rng, 1, 64)
        high = _log(rng, 1, 92160)
        new_high = _log(rng, 1, 2048)
        return dict(op=op, S=S, low=rng.randint(0, high), high=high, new_low=rng.randint(0, new_high), new_high=new_high,
                    page=rng.choice([1, 16, 32, 64]), maps=rng.random() < 0.6, pad=rng.choice([0, 1, 77, 1024]))
    if op == "store":
        Hkv, D, dtype = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.choice(["bf16", "f32"])
        most = (1 << 25) // (Hkv * D) // (1 if dtype == "bf16" else 2)
        return dict(op=op, T=_log(rng, 1, min(32768, most)), Hkv=Hkv, D=D, page=rng.choice([1, 16, 32, 64]), dtype=dtype,
                    fused=rng.random() < 0.5, skip=rng.choice([0.0, 0.1]))
    if op == "decode":
        S, Tq, G = _log(rng, 1, 36), rng.choice([1, 1, 1, 2, 4, 7]), rng.randint(1, 8)
        Hkv, D, maps = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.random() < 0.5
        most = (1 << 28) // (S * Hkv * D) // max(1, Tq * G // 8)
        high = _log(rng, 1, min(92160, most))
        return dict(op=op, S=S, Tq=Tq, Hq=Hkv * G, Hkv=Hkv, D=D, low=rng.randint(1, high), high=high,
                    page=rng.choice([1, 16, 32, 64]), maps=maps, live=rng.choice([0.1, 0.25, 0.9, 1.0]) if maps else 1.0)
    S = _log(rng, 1, 16)
    T = _log(rng, S, 12000)
    Hkv = rng.choice([1, 2, 4, 8])
    return dict(op=op, S=S, T=T, low=rng.randint(0, T // S), Hq=Hkv * rng.randint(1, 5), Hkv=Hkv, D=rng.choice([64, 128]),
                fused=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _spread(low, high, n):
    """n lengths from low to high in even steps: their sum is the case's, the seed shuffles them."""
    if n == 1:
        return [high]
    return [low + (high - low) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """The lengths of a case's sessions or sequences, in no order."""
    if case["op"] == "prompt":
        # they add up to T and grow about quadratically from `low`
        S, T, low = case["S"], case["T"], case["low"]
        if S == 1:
            return [T]
        weights = [i * i for i in range(S)]
        total, rest = sum(weights), T - low * S
        lens = [low + rest * w // total for w in weights]
        lens[-1] += T - sum(lens)
        return lens
    return _spread(case["low"], case["high"], case["S"])


def _shuffled(lens, g):
    order = torch.randperm(len(lens), generator=g, device=DEVICE)
    return torch.tensor(lens, dtype=torch.int32, device=DEVICE)[order].contiguous()


def _keys(shape, g):
    """Rows as a cache sees them: normal values with a few channels eight times as large."""
    x = torch.randn(shape, generator=g, device=DEVICE)
    big = torch.rand(shape[-2:], generator=g, device=DEVICE) < 0.02
    return x * torch.where(big, 8.0, 1.0)


def _empty_cache(P, Hkv, page, D):
    return (torch.zeros((P, Hkv, page, D // 2), dtype=torch.uint8, device=DEVICE),
            torch.zeros((P, Hkv, page, D // GROUP), dtype=torch.uint8, device=DEVICE))


def _filled_cache(P, Hkv, page, D, g, outliers):
    codes, scales = _empty_cache(P, Hkv, page, D)
    step = max(1, (1 << 25) // (Hkv * page * D))
    for p in range(0, P, step):
        n = min(step, P - p)
        shape = (n * page, Hkv, D)
        x = (_keys(shape, g) if outliers else torch.randn(shape, generator=g, device=DEVICE)).to(torch.bfloat16)
        c, s = _quantise(x.view(n, page, Hkv, D).permute(0, 2, 1, 3))
        codes[p:p + n], scales[p:p + n] = c, s
    return codes, scales


def prepare(case, seed):
    g = _generator(seed)
    st, op = dict(case=case), case["op"]
    if op == "plan":
        S, page = case["S"], case["page"]
        cached = _shuffled(_lengths(case), g)
        new = _shuffled(_spread(case["new_low"], case["new_high"], S), g)
        rows = -(-(case["high"] + case["new_high"]) // page)
        T = sum(_spread(case["new_low"], case["new_high"], S)) + case["pad"]
        P = S * rows
        perm = torch.randperm(P, generator=g, device=DEVICE).to(torch.int32)
        table = perm.view(S, rows).clone()
        have = (cached + page - 1) // page
        table[torch.arange(rows, device=DEVICE)[None] >= have[:, None]] = -1
        taken = torch.zeros(P, dtype=torch.bool, device=DEVICE)
        taken[table[table >= 0].long()] = True
        free = perm.flip(0)[~taken[perm.flip(0).long()]].contiguous()
        st.update(cached=cached, new=new, table=table, free=free, P=P, T=T,
                  cu=torch.empty(S + 1, dtype=torch.int32, device=DEVICE),
                  slots=torch.empty(T, dtype=torch.int32, device=DEVICE),
                  pos=torch.empty(T, dtype=torch.int32, device=DEVICE),
                  counts=torch.empty(2, dtype=torch.int32, device=DEVICE),
                  map=torch.empty((S, rows * page), dtype=torch.int32, device=DEVICE) if case["maps"] else None)
    elif op == "store":
        T, Hkv, D, page = case["T"], case["Hkv"], case["D"], case["page"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        k, v = _keys((T, Hkv, D), g).to(dt), torch.randn((T, Hkv, D), generator=g, device=DEVICE).to(dt)
        if case["fused"]:  # slices of one projection's output [T][(Hkv + Hkv) D]
            both = torch.cat([k.view(T, -1), v.view(T, -1)], dim=1)
            k, v = both[:, :Hkv * D].view(T, Hkv, D), both[:, Hkv * D:].view(T, Hkv, D)
        P = -(-T // page) + 3
        pages = torch.randperm(P, generator=g, device=DEVICE)
        t = torch.arange(T, device=DEVICE)
        slots = (pages[t // page] * page + t % page).to(torch.int32)
        slots[torch.rand(T, generator=g, device=DEVICE) < case["skip"]] = -1
        kc, ks = _empty_cache(P, Hkv, page, D)
        vc, vs = _empty_cache(P, Hkv, page, D)
        st.update(k=k, v=v, slots=slots, kc=kc, ks=ks, vc=vc, vs=vs,
                  k_back=torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEVICE),
                  v_back=torch.empty((T, Hkv, D), dtype=torch.bfloat16, device=DEVICE))
    elif op == "decode":
        S, Tq, Hq, Hkv, D, page = (case[x] for x in ("S", "Tq", "Hq", "Hkv", "D", "page"))
        lens = _shuffled(_lengths(case), g)
        rows = -(-case["high"] // page)
        q = torch.randn((S, Tq, Hq, D), generator=g, device=DEVICE).to(torch.bfloat16)
        j = torch.arange(rows * page, device=DEVICE)
        if case["maps"]:  # the kept tokens of each session in pages of their own, the dropped ones at the dead slot
            kept = (torch.rand((S, rows * page), generator=g, device=DEVICE) < case["live"]) | (j[None] < 16)
            kept &= j[None] < lens[:, None]
            rank = kept.long().flatten().cumsum(0).view(S, -1) - 1
            P = -(-max(1, int(kept.sum())) // page) + 1
            pages = torch.randperm(P, generator=g, device=DEVICE)
            at = rank.clamp(min=0)
            slot_map = torch.where(kept, pages[at // page] * page + at % page, P * page).to(torch.int32)
            st.update(slot_map=slot_map.contiguous(), table=None, dead=P * page)
        else:
            P = S * rows
            table = torch.randperm(P, generator=g, device=DEVICE).to(torch.int32).view(S, rows)
            st.update(slot_map=None, table=table.contiguous(), dead=None)
        kc, ks = _filled_cache(P, Hkv, page, D, g, True)
        vc, vs = _filled_cache(P, Hkv, page, D, g, False)
        st.update(q=q, lens=lens, kc=kc, ks=ks, vc=vc, vs=vs, scale=D ** -0.5, out=torch.empty_like(q),
                  lse=torch.empty((S, Tq, Hq), dtype=torch.float32, device=DEVICE))
    else:
        T, Hq, Hkv, D = (case[x] for x in ("T", "Hq", "Hkv", "D"))
        lens = _shuffled(_lengths(case), g)
        cu = torch.zeros(case["S"] + 1, dtype=torch.int32, device=DEVICE)
        cu[1:] = lens.cumsum(0)
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEVICE).to(torch.bfloat16)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if not case["fused"]:
            q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        st.update(q=q, k=k, v=v, cu=cu, longest=max(_lengths(case)), scale=D ** -0.5,
                  out=torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEVICE),
                  lse=torch.empty((T, Hq), dtype=torch.float32, device=DEVICE))
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _scale_values(dtype):
    """The value of each scale byte up to the largest in use."""
    bits = (torch.arange(TOP_BYTE + 1, device=DEVICE, dtype=torch.int32) << 7).to(torch.int16)
    return bits.view(torch.float16).to(dtype)


def _quantise(x):
    """[..., D] values -> codes [..., D/2] and scales [..., D/16], both uint8."""
    grp = x.float().unflatten(-1, (-1, GROUP))
    mag = grp.abs()
    top = mag.amax(-1, keepdim=True)                            # a NaN in the group comes out as NaN
    steps = _scale_values(torch.float32)
    byte = torch.searchsorted(steps * 6, top.contiguous())      # 6 * scale is exact: the first that reaches the largest value
    broken = ~(top <= 61440.0)
    byte = torch.where(broken, TOP_BYTE, byte)
    s = steps[byte]
    code = torch.zeros_like(mag, dtype=torch.uint8)
    for border, up in BORDERS:                                  # border * scale is exact
        code += (mag >= border * s) & (s > 0) if up else mag > border * s
    code |= torch.signbit(grp).to(torch.uint8) << 3
    code = torch.where(broken, 0, code).flatten(-2)
    byte = torch.where(broken, 255, byte).squeeze(-1).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte


def _dequantise(codes, scales):
    """The fp32 values of codes [..., D/2] and scales [..., D/16]."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=DEVICE)
    nib = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2)
    s = (scales.to(torch.int32) << 7).to(torch.int16).view(torch.float16).float()
    return (table[nib.int()].unflatten(-1, (-1, GROUP)) * s.unsqueeze(-1)).flatten(-2)


def _plan(st):
    case, cached, new, table, free = st["case"], st["cached"], st["new"], st["table"], st["free"]
    page, T, S = case["page"], st["T"], case["S"]
    have, need = (cached + page - 1) // page, (cached + new + page - 1) // page
    take = need - have
    before = take.cumsum(0) - take
    j = torch.arange(table.shape[1], device=DEVICE)[None]
    fresh = (j >= have[:, None]) & (j < need[:, None])
    source = (before[:, None] + j - have[:, None]).clamp(0, max(0, free.numel() - 1))
    if free.numel():
        table.copy_(torch.where(fresh, free[source], table))
    cu = torch.zeros(S + 1, dtype=torch.int32, device=DEVICE)
    cu[1:] = new.cumsum(0)
    i = torch.arange(T, device=DEVICE, dtype=torch.int32)
    s = torch.searchsorted(cu[1:].contiguous(), i, right=True)
    real = s < S
    s = s.clamp(max=S - 1)
    pos = cached[s] + i - cu[s]
    slot = table[s, torch.where(real, pos // page, 0)] * page + pos % page
    slots = torch.where(real, slot, -1).to(torch.int32)
    pos = torch.where(real, pos, -1).to(torch.int32)
    counts = torch.stack([cu[S], take.sum()]).to(torch.int32)
    out = dict(table=table, cu=cu, slots=slots, pos=pos, counts=counts)
    if case["maps"]:
        p = torch.arange(table.shape[1] * page, device=DEVICE)
        every = table[:, p // page] * page + p % page
        out["map"] = torch.where(p[None] < (cached + new)[:, None], every, -1).to(torch.int32)
    return out


def _store(st):
    P, Hkv, page, _ = st["kc"].shape
    slots = st["slots"].long()
    real = slots >= 0
    # a token without a slot writes what the first token that has one writes, to the same place
    stand = torch.where(real, torch.arange(slots.numel(), device=DEVICE), real.int().argmax())
    spare = slots[stand].clamp(min=0)
    head = torch.arange(Hkv, device=DEVICE)[None]
    at, off = (spare // page)[:, None], (spare % page)[:, None]
    back, some, real = [], real.any(), real[:, None, None]
    for x, codes, scales in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
        c, s = _quantise(x)
        codes[at, head, off] = torch.where(some, c[stand], codes[at, head, off])
        scales[at, head, off] = torch.where(some, s[stand], scales[at, head, off])
        back.append(torch.where(real, _dequantise(codes[at, head, off], scales[at, head, off]), 0.0).to(torch.bfloat16))
    return dict(k=back[0], v=back[1])


def _decode(st):
    case, q, lens = st["case"], st["q"].float(), st["lens"]
    S, Tq, Hq, Hkv, D, page = (case[x] for x in ("S", "Tq", "Hq", "Hkv", "D", "page"))
    if st["slot_map"] is not None:
        slots, live = st["slot_map"], st["slot_map"] != st["dead"]
    else:
        j = torch.arange(st["table"].shape[1] * page, device=DEVICE)
        slots = st["table"][:, j // page] * page + j % page
        live = torch.ones_like(slots, dtype=torch.bool)
    N = slots.shape[1]
    at = torch.where(live, slots, 0).long()
    j = torch.arange(N, device=DEVICE)

    def rows(codes, scales):  # [S][Hkv][N][D]
        h = torch.arange(Hkv, device=DEVICE)[None, :, None]
        p, o = (at // page)[:, None], (at % page)[:, None]
        return _dequantise(codes[p, h, o], scales[p, h, o])

    G = Hq // Hkv
    qs = q.view(S, Tq, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(S, Hkv, Tq * G, D)
    x = torch.matmul(qs, rows(st["kc"], st["ks"]).transpose(-1, -2)) * st["scale"]
    pos = lens[:, None] - Tq + torch.arange(Tq, device=DEVICE)[None]
    seen = live[:, None] & (j[None, None] <= pos[:, :, None])                       # [S][Tq][N]
    seen = seen.repeat_interleave(G, dim=1)[:, None]                                 # [S][1][Tq G][N]
    out, lse = _softmax_product(x, seen, lambda: rows(st["vc"], st["vs"]))
    out = out.view(S, Hkv, Tq, G, D).permute(0, 2, 1, 3, 4).reshape(S, Tq, Hq, D)
    lse = lse.view(S, Hkv, Tq, G).permute(0, 2, 1, 3).reshape(S, Tq, Hq)
    return dict(out=out.to(torch.bfloat16), lse=lse)


def _softmax_product(x, seen, values):
    """Rows of softmax(x over seen places) times values(); (rows, log of the sum); zero and -inf where nothing is seen."""
    x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    base = torch.where(top == -math.inf, 0.0, top)
    x.sub_(base).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x, values()) / torch.where(total == 0, 1.0, total)
    return out, (base + total.log()).squeeze(-1)


def _prompt(st):
    case, cu = st["case"], st["cu"].long()
    S, T, Hq, Hkv, D = (case[x] for x in ("S", "T", "Hq", "Hkv", "D"))
    n, G = st["longest"], Hq // Hkv
    i = torch.arange(n, device=DEVICE)
    inside = i[None] < (cu[1:] - cu[:-1])[:, None]                                   # [S][n]
    at = torch.where(inside, cu[:-1, None] + i[None], 0)

    def padded(x):  # [S][Hkv][heads of the group][n][D]
        return x.float()[at].view(S, n, Hkv, -1, D).permute(0, 2, 3, 1, 4)

    x = torch.matmul(padded(st["q"]), padded(st["k"]).transpose(-1, -2)).mul_(st["scale"])
    seen = i[None, :] <= i[:, None]
    out, lse = _softmax_product(x, seen, lambda: padded(st["v"]))
    s = torch.searchsorted(cu[1:].contiguous(), torch.arange(T, device=DEVICE), right=True)
    where = s * n + torch.arange(T, device=DEVICE) - cu[s]                            # each token's place among the padded
    out = out.permute(0, 3, 1, 2, 4).reshape(S * n, Hq, D)[where]
    lse = lse.permute(0, 3, 1, 2).reshape(S * n, Hq)[where]
    return dict(out=out.to(torch.bfloat16), lse=lse)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

_kept = []


def _context():
    """The program's one context, made by its first call."""
    if not _kept:
        import kv_cache_retention_gb300 as kv
        _kept.append(kv.Context(0))
    return _kept[0]


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"plan": _plan, "store": _store, "decode": _decode, "prompt": _prompt}[op](st)
    ctx = _context()
    if op == "plan":
        ctx.plan_slots(st["cached"], st["new"], st["free"], st["case"]["page"], st["P"], st["table"], st["cu"],
                       st["slots"], st["pos"], st["counts"], slot_map=st["map"])
        out = dict(table=st["table"], cu=st["cu"], slots=st["slots"], pos=st["pos"], counts=st["counts"])
        return out if st["map"] is None else dict(out, map=st["map"])
    if op == "store":
        ctx.kv4_store(st["k"], st["v"], st["slots"], st["kc"], st["ks"], st["vc"], st["vs"])
        ctx.kv4_load(st["kc"], st["ks"], st["vc"], st["vs"], st["slots"], st["k_back"], st["v_back"])
        return dict(k=st["k_back"], v=st["v_back"])
    if op == "decode":
        ctx.kv4_attention(st["q"], st["kc"], st["ks"], st["vc"], st["vs"], st["lens"], st["out"], scale=st["scale"],
                          slot_map=st["slot_map"], block_table=st["table"], dead_slot=st["dead"], lse=st["lse"])
        return dict(out=st["out"], lse=st["lse"])
    ctx.prompt_attention(st["q"], st["k"], st["v"], st["cu"], st["out"], scale=st["scale"], lse=st["lse"])
    return dict(out=st["out"], lse=st["lse"])


def work(case):
    op = case["op"]
    if op == "plan":
        S, page = case["S"], case["page"]
        new = sum(_spread(case["new_low"], case["new_high"], S))
        cached = sum(_lengths(case))
        rows = -(-(case["high"] + case["new_high"]) // page)
        table = (cached + new) / page if case["maps"] else new / page + S
        maps = S * rows * page if case["maps"] else 0
        return dict(bytes=4 * (2 * S + S + 1 + 2 * (new + case["pad"]) + 2 * new / page + table + maps), flops=0)
    if op == "store":
        T, Hkv, D = case["T"], case["Hkv"], case["D"]
        rows = 2 * T * Hkv * (1 - case["skip"])
        one = D // 2 + D // GROUP
        size = 2 if case["dtype"] == "bf16" else 4
        # written from the rows, then read back into bf16 rows
        return dict(bytes=rows * (D * size + one) + rows * one + 2 * T * Hkv * D * 2 + 8 * T, flops=0)
    if op == "decode":
        S, Tq, Hq, Hkv, D = (case[x] for x in ("S", "Tq", "Hq", "Hkv", "D"))
        tokens = sum(_lengths(case))
        live = tokens * case["live"]
        ids = 4 * tokens if case["maps"] else 4 * tokens / case["page"]
        return dict(bytes=2 * live * Hkv * (D // 2 + D // GROUP) + ids + 4 * S * Tq * Hq * D + 4 * S * Tq * Hq,
                    flops=4 * live * Tq * Hq * D)
    T, Hq, Hkv, D = (case[x] for x in ("T", "Hq", "Hkv", "D"))
    pairs = sum(n * (n + 1) // 2 for n in _lengths(case))
    return dict(bytes=2 * T * D * (2 * Hq + 2 * Hkv) + 4 * T * Hq, flops=4 * pairs * Hq * D)


# ---------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------

def _value_of(codes, scales):
    """64-bit values of stored groups, from the format's definition: sign, exponent and mantissa fields."""
    pair = torch.stack((codes.bitwise_and(0x0F), codes.bitwise_right_shift(4)), -1).reshape(*codes.shape[:-1], -1).long()
    e, m = (pair >> 1) & 3, (pair & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, e.double() - 1))
    val = torch.where(pair >= 8, -mag, mag)
    b = scales.long()
    be, bm = b >> 3, (b & 7).double()
    sc = torch.where(be == 0, bm * 2.0 ** -17, (1 + bm / 8) * torch.pow(2.0, be.double() - 15))
    sc = torch.where(b == 255, math.nan, sc)
    return val * sc.repeat_interleave(GROUP, dim=-1)


def _exact_store(st):
    out = {}
    ladder = torch.tensor(sorted({(1 + m / 8) * 2.0 ** (e - 15) for e in range(1, 29) for m in range(8)
                                  if (1 + m / 8) * 2.0 ** (e - 15) <= 10240} | {m * 2.0 ** -17 for m in range(8)}),
                          dtype=torch.float64, device=DEVICE)
    levels = torch.tensor(MAGNITUDES, dtype=torch.float64, device=DEVICE)
    odd = torch.tensor([0, 1, 0, 1, 0, 1, 0, 1], dtype=torch.float64, device=DEVICE)
    for name in ("k", "v"):
        parts = []
        for x in st[name].split(2048):
            x = x.double().unflatten(-1, (-1, GROUP))
            top = x.abs().amax(-1)
            s = ladder[torch.searchsorted(ladder, (top / 6).contiguous()).clamp(max=ladder.numel() - 1)]
            s = torch.where(s * 6 < top, ladder[(torch.searchsorted(ladder, s) + 1).clamp(max=ladder.numel() - 1)], s)
            y = x.abs() / torch.where(s > 0, s, 1.0).unsqueeze(-1)
            away = (y.unsqueeze(-1) - levels).abs()
            least = away.amin(-1, keepdim=True)
            # of the (at most two) nearest levels, the even one
            pick = torch.where(away == least, odd, 9.0).argmin(-1)
            parts.append((levels[pick] * torch.sign(x) * s.unsqueeze(-1)).flatten(-2))
        val = torch.cat(parts)
        val[st["slots"] < 0] = 0
        out[name] = val
    return out


def _exact_rows(q, k, v, scale, first):
    """One kv head: q [R][D] rows, row r over keys [0, first[r]]; -> rows and log-sums in 64 bits."""
    x = q @ k.T * scale
    x[torch.arange(k.shape[0], device=DEVICE)[None] > first[:, None]] = -math.inf
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    return p @ v, lse


def _exact_decode(st):
    case = st["case"]
    S, Tq, Hq, Hkv, D, page = (case[x] for x in ("S", "Tq", "Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    out = torch.zeros((S, Tq, Hq, D), dtype=torch.float64, device=DEVICE)
    lse = torch.full((S, Tq, Hq), -math.inf, dtype=torch.float64, device=DEVICE)
    for s in range(S):
        n = int(st["lens"][s])
        if st["slot_map"] is not None:
            slot = st["slot_map"][s, :n].long()
            where = torch.nonzero(slot != st["dead"]).flatten()
            slot = slot[where]
        else:
            where = torch.arange(n, device=DEVICE)
            slot = st["table"][s].long().repeat_interleave(page)[:n] * page + where % page
        if not where.numel():
            continue
        # the last key each query row sees, as an index among the live ones
        pos = n - Tq + torch.arange(Tq, device=DEVICE)
        last = torch.searchsorted(where, pos, right=True) - 1
        for h in range(Hkv):
            k = _value_of(st["kc"][slot // page, h, slot % page], st["ks"][slot // page, h, slot % page])
            v = _value_of(st["vc"][slot // page, h, slot % page], st["vs"][slot // page, h, slot % page])
            q = st["q"][s, :, h * G:(h + 1) * G].double().reshape(Tq * G, D)
            o, l = _exact_rows(q, k, v, st["scale"], last.repeat_interleave(G))
            out[s, :, h * G:(h + 1) * G] = torch.where(torch.isinf(l)[:, None], 0.0, o).view(Tq, G, D)
            lse[s, :, h * G:(h + 1) * G] = l.view(Tq, G)
    return dict(out=out, lse=lse)


def _exact_prompt(st):
    case = st["case"]
    T, Hq, Hkv, D = (case[x] for x in ("T", "Hq", "Hkv", "D"))
    out = torch.empty((T, Hq, D), dtype=torch.float64, device=DEVICE)
    lse = torch.empty((T, Hq), dtype=torch.float64, device=DEVICE)
    edges = st["cu"].tolist()
    for a, b in zip(edges[:-1], edges[1:]):
        for h in range(Hq):
            k, v = st["k"][a:b, h * Hkv // Hq].double(), st["v"][a:b, h * Hkv // Hq].double()
            for r in range(a, b, 4096):
                e = min(b, r + 4096)
                out[r:e, h], lse[r:e, h] = _exact_rows(st["q"][r:e, h].double(), k[:e - a], v[:e - a], st["scale"],
                                                       torch.arange(r - a, e - a, device=DEVICE))
    return dict(out=out, lse=lse)


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    st = prepare(case, seed)
    return {"store": _exact_store, "decode": _exact_decode, "prompt": _exact_prompt}[case["op"]](st)
