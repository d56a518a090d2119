"""Attention over the paged K/V pools, the weight it gives to each cached token, and eviction by that weight, each in its
plain form and as the library's call.

  attend  pool_attention: attention of packed new tokens (one to thousands for each session) over the bf16 page pools
  mass    attention_mass: the softmax weight that the new tokens give to each token of their session, added to a score
  evict   evict_slots: the tokens of least score leave the slot maps of sessions above their budget, their slots are listed

``run`` computes a case's operator in elementary torch operations while ``own`` is false, and with the calls of
kv_cache_retention_gb300 while it is true.

New tokens are packed: session s has the tokens [cu[s], cu[s+1]) of q, the last of its lens[s] tokens, so token i of them
sits at position lens[s] - new + i and sees the tokens j up to its own whose slot is live.  Slots come from slot maps,
in which dropped tokens point at the dead slot, or from block tables.  Pools are [P][page][Hkv][D].
"""
import math
import random

import torch

own = False

DEVICE = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the smallest call: one decode step of one session of a small model
        dict(name="attend tiny", op="attend", S=1, new_low=1, new_high=1, low=2048, high=2048, Hq=4, Hkv=2, D=64, page=16,
             maps=False, live=1.0, fused=False),
        # a decode step of 36 sessions after pruning to a quarter: slot maps whose dropped tokens point at the dead slot
        dict(name="attend decode pruned 36", op="attend", S=36, new_low=1, new_high=1, low=20000, high=32768, Hq=32, Hkv=8,
             D=128, page=16, maps=True, live=0.25, fused=True),
        # a decode step of one long session, groups of five heads
        dict(name="attend decode long 92160", op="attend", S=1, new_low=1, new_high=1, low=92160, high=92160, Hq=40, Hkv=8,
             D=128, page=32, maps=False, live=1.0, fused=False),
        # one step of a serving batch that mixes decode steps with chunks of prompts, uneven and odd lengths
        dict(name="attend mixed 16", op="attend", S=16, new_low=1, new_high=1013, low=1301, high=16384, Hq=32, Hkv=8, D=128,
             page=16, maps=True, live=0.9, fused=True),
        # a chunk of a long prompt: 2048 tokens behind 32768 cached ones
        dict(name="attend chunk 2048", op="attend", S=1, new_low=2048, new_high=2048, low=34816, high=34816, Hq=32, Hkv=8,
             D=128, page=16, maps=False, live=1.0, fused=True),
        # a follow-up question of a small model, odd sizes, groups of seven heads
        dict(name="attend turn 333", op="attend", S=3, new_low=77, new_high=333, low=1999, high=7777, Hq=14, Hkv=2, D=64,
             page=32, maps=True, live=0.5, fused=True),
        # the smallest scoring call: one decode step
        dict(name="mass tiny", op="mass", S=1, new_low=1, new_high=1, low=2048, high=2048, Hq=4, Hkv=2, D=64, page=16,
             maps=True, live=1.0, fused=False),
        # the weights of a decode step of 36 sessions, added to what the earlier steps gave
        dict(name="mass decode pruned 36", op="mass", S=36, new_low=1, new_high=1, low=20000, high=32768, Hq=32, Hkv=8, D=128,
             page=16, maps=True, live=0.25, fused=True),
        # the weights that a chunk of a long prompt gives to everything before it
        dict(name="mass chunk 2048", op="mass", S=1, new_low=2048, new_high=2048, low=34816, high=34816, Hq=32, Hkv=8, D=128,
             page=16, maps=False, live=1.0, fused=True),
        # 36 sessions at their budget: each gained a token and gives one up
        dict(name="evict step 36", op="evict", S=36, low=5000, high=8192, live=0.5, over=1, freed=1),
        # one long session cut down to a tenth after its prompt
        dict(name="evict long 92160", op="evict", S=1, low=92160, high=92160, live=1.0, over=82944, freed=92160),
        # 64 long sessions cut down by a quarter of their live tokens
        dict(name="evict 64 long", op="evict", S=64, low=1, high=92160, live=0.8, over=18432, freed=92160),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "mass", "evict"])
    if op == "evict":
        S = _log(rng, 1, 64)
        high = _log(rng, 1, 92160)
        return dict(op=op, S=S, low=rng.randint(0, high), high=high, live=rng.choice([0.1, 0.5, 0.9, 1.0]),
                    over=_log(rng, 1, high), freed=rng.choice([1, 64, high]))
    D, Hkv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.randint(1, 8)
    S = _log(rng, 1, 36)
    # tokens and products of a call stay below those of the largest cases
    high = _log(rng, 1, min(92160, (1 << 28) // (S * Hkv * D)))
    new = _log(rng, 1, max(1, min(2048, high, (1 << 31) // (S * high * Hq), (1 << 18) // (S * Hq))))
    maps = rng.random() < 0.5
    return dict(op=op, S=S, new_low=rng.randint(1, new), new_high=new, low=rng.randint(min(new, high), high), high=high, Hq=Hq,
                Hkv=Hkv, D=D, page=rng.choice([1, 16, 32, 64]), maps=maps, live=rng.choice([0.1, 0.5, 0.9, 1.0]) if maps else 1.0,
                fused=rng.random() < 0.5)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _spread(low, high, n):
    """n whole numbers from low to high in even steps."""
    return [high] if n == 1 else [low + (high - low) * i // (n - 1) for i in range(n)]


def _sessions(case):
    """(new tokens, length) of each session, the longest with the fewest new tokens."""
    lens = _spread(case["low"], case["high"], case["S"])
    new = _spread(case["new_low"], case["new_high"], case["S"])
    return [(min(m, n), n) for m, n in zip(reversed(new), lens)]


def _shuffled(values, seed):
    values = list(values)
    random.Random(seed).shuffle(values)
    return values


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _keys(shape, g):
    """Rows as a cache sees them: normal values with a few channels eight times as large."""
    big = torch.rand(shape[-2:], generator=g, device=DEVICE) < 0.02
    return torch.randn(shape, generator=g, device=DEVICE).mul_(torch.where(big, 8.0, 1.0))


def _pages(lens, page, share, protect, g):
    """Slot maps [S][positions] of sessions with pages of their own, and the number of pages.  A share of the tokens is
    live (the first four and the last `protect[s]` of a session all are); kept rows have stayed where they were."""
    S, rows = len(lens), -(-max(lens) // page)
    j, size = torch.arange(rows * page, device=DEVICE), _int32(lens)[:, None]
    live = (torch.rand((S, rows * page), generator=g, device=DEVICE) < share) | (j < 4) | (j >= size - _int32(protect)[:, None])
    P = S * rows
    table = torch.randperm(P, generator=g, device=DEVICE).view(S, rows)
    slots = torch.where(live & (j < size), table[:, j // page] * page + j % page, P * page)
    return slots.to(torch.int32).contiguous(), P


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    S = case["S"]
    st = dict(case=case)
    if case["op"] == "evict":
        lens = _shuffled(_spread(case["low"], case["high"], S), seed)
        st["lens"] = _int32(lens)
        slots, P = _pages([max(1, n) for n in lens], 16, case["live"], [0] * S, g)
        st["dead"] = P * 16
        n = slots.shape[1]
        j = torch.arange(n, device=DEVICE)
        slots = torch.where(j[None] < st["lens"][:, None], slots, -1)
        have = ((slots >= 0) & (slots != st["dead"])).sum(1)
        # sums of softmax weights: a few large ones, a long tail, and tokens that nothing has looked at yet
        score = torch.randn((S, n), generator=g, device=DEVICE).mul_(2.5).exp_()
        score = torch.where(torch.rand((S, n), generator=g, device=DEVICE) < 0.05, 0.0, score)
        st.update(slots=slots.contiguous(), score=score.contiguous(), sink=4, recent=32,
                  budget=(have - case["over"]).clamp(min=0).to(torch.int32), out=torch.empty_like(slots),
                  freed=torch.empty((S, case["freed"]), dtype=torch.int32, device=DEVICE),
                  n_freed=torch.empty(S, dtype=torch.int32, device=DEVICE))
        return st
    Hq, Hkv, D, page = (case[x] for x in ("Hq", "Hkv", "D", "page"))
    new, lens = zip(*_shuffled(_sessions(case), seed))
    st.update(lens_host=lens, lens=_int32(lens))
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    T = cu[-1]
    if case["maps"]:
        slots, P = _pages(lens, page, case["live"], new, g)
        st.update(slots=slots, table=None, dead=P * page)
    else:
        rows = -(-max(lens) // page)
        P = S * rows
        st.update(slots=None, table=torch.randperm(P, generator=g, device=DEVICE).to(torch.int32).view(S, rows).contiguous(),
                  dead=None)
    rows = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEVICE).to(torch.bfloat16)  # a fused projection's output
    q = rows[:, :Hq] if case["fused"] else rows[:, :Hq].contiguous()
    st.update(new_host=new, cu_host=cu, cu=_int32(cu), q=q, scale=D ** -0.5,
              k_pool=_keys((P, page, Hkv, D), g).to(torch.bfloat16))
    if case["op"] == "attend":
        st.update(v_pool=torch.randn((P, page, Hkv, D), generator=g, device=DEVICE).to(torch.bfloat16),
                  out=torch.empty((T, Hq, D), dtype=torch.bfloat16, device=DEVICE),
                  lse=torch.empty((T, Hq), dtype=torch.float32, device=DEVICE))
    else:
        st["lse"] = torch.cat([_log_sum(_logits(st, s)) for s in range(S)])
        n = st["slots"].shape[1] if case["maps"] else st["table"].shape[1] * page
        st.update(before=torch.randn((S, n), generator=g, device=DEVICE).exp_(),
                  score=torch.empty((S, n), dtype=torch.float32, device=DEVICE))
    return st


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------

def _session_slots(st, s):
    """Slots of session s's positions (0 where the token is not live), and which are live."""
    n = st["lens_host"][s]
    if st["slots"] is not None:
        slots = st["slots"][s, :n]
        live = (slots >= 0) & (slots != st["dead"])
        return torch.where(live, slots, 0).long(), live
    j, page = torch.arange(n, device=DEVICE), st["case"]["page"]
    return st["table"][s].long()[j // page] * page + j % page, torch.ones(n, dtype=torch.bool, device=DEVICE)


def _rows_of(pool, slots):
    return pool.flatten(0, 1)[slots].float().transpose(0, 1)                     # [Hkv][n][D]


def _logits(st, s):
    """Session s's logits [Hkv][new][heads of the group][n] in fp32, -inf where a token is not seen."""
    case, (slots, live) = st["case"], _session_slots(st, s)
    Hkv, D, n, m = case["Hkv"], case["D"], st["lens_host"][s], st["new_host"][s]
    q = st["q"][st["cu_host"][s]:st["cu_host"][s + 1]].float().view(m, Hkv, -1, D).transpose(0, 1)
    x = torch.matmul(q.flatten(1, 2), _rows_of(st["k_pool"], slots).transpose(1, 2)).mul_(st["scale"]).view(Hkv, m, -1, n)
    j = torch.arange(n, device=DEVICE)
    seen = live[None] & (j[None] <= j[n - m:, None])
    return x.masked_fill_(~seen[:, None], -math.inf)


def _log_sum(x):
    """The log of the sum of e^x, [new][Hq], of _logits' result."""
    top = x.amax(-1)
    base = torch.where(top == -math.inf, 0.0, top)
    total = torch.exp(x - base[..., None]).sum(-1)
    return (base + total.log()).transpose(0, 1).flatten(1)


def _attend(st):
    case = st["case"]
    out, lse = [], []
    for s in range(case["S"]):
        x = _logits(st, s)
        top = x.amax(-1, keepdim=True)
        base = torch.where(top == -math.inf, 0.0, top)
        p = x.sub_(base).exp_()
        total = p.sum(-1, keepdim=True)
        slots, live = _session_slots(st, s)
        v = torch.where(live[None, :, None], _rows_of(st["v_pool"], slots), 0.0)
        o = torch.matmul(p.flatten(1, 2), v).view(*p.shape[:3], -1) / torch.where(total == 0, 1.0, total)
        out.append(o.transpose(0, 1).flatten(1, 2).to(torch.bfloat16))
        lse.append((base + total.log()).squeeze(-1).transpose(0, 1).flatten(1))
    return dict(out=torch.cat(out), lse=torch.cat(lse))


def _mass(st):
    case = st["case"]
    score = st["before"].clone()
    for s in range(case["S"]):
        n, a, b = st["lens_host"][s], st["cu_host"][s], st["cu_host"][s + 1]
        lse = st["lse"][a:b].view(b - a, case["Hkv"], -1).transpose(0, 1)[..., None]
        p = _logits(st, s).sub_(lse).exp_()
        p = torch.where(lse == -math.inf, 0.0, p)
        score[s, :n] += p.sum((0, 1, 2))
    return dict(score=score)


def _evict(st):
    slots, score, lens = st["slots"], st["score"], st["lens"].long()[:, None]
    n, room = slots.shape[1], st["freed"].shape[1]
    j = torch.arange(n, device=DEVICE)[None]
    live = (j < lens) & (slots >= 0) & (slots != st["dead"])
    free = live & (j >= st["sink"]) & (j < lens - st["recent"])
    leave = torch.minimum(live.sum(1) - st["budget"], free.sum(1)).clamp(0, room)
    # the least scores leave; of equal ones the later position
    value = torch.where(free, score + 0.0, math.inf).flip(1)
    order = torch.sort(value, dim=1, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order).contiguous()).flip(1)
    gone = rank < leave[:, None]
    at = torch.where(gone, gone.long().cumsum(1) - 1, room)
    freed = torch.full((slots.shape[0], room + 1), -1, dtype=torch.int32, device=DEVICE)
    freed.scatter_(1, at, slots)
    return dict(slots=torch.where(gone, st["dead"], slots), freed=freed[:, :room], n_freed=leave.to(torch.int32))


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
        return {"attend": _attend, "mass": _mass, "evict": _evict}[op](st)
    ctx = _context()
    if op == "attend":
        ctx.pool_attention(st["q"], st["k_pool"], st["v_pool"], st["cu"], st["lens"], st["out"], slot_map=st["slots"],
                           block_table=st["table"], dead_slot=st["dead"], scale=st["scale"], lse=st["lse"])
        return dict(out=st["out"], lse=st["lse"])
    if op == "mass":
        ctx.attention_mass(st["q"], st["lse"], st["k_pool"], st["cu"], st["lens"], st["score"], slot_map=st["slots"],
                           block_table=st["table"], dead_slot=st["dead"], scale=st["scale"], score_in=st["before"])
        return dict(score=st["score"])
    ctx.evict_slots(st["score"], st["lens"], st["budget"], st["slots"], st["dead"], st["out"], n_sink=st["sink"],
                    n_recent=st["recent"], freed=st["freed"], n_freed=st["n_freed"])
    return dict(slots=st["out"], freed=st["freed"], n_freed=st["n_freed"])


def work(case):
    S = case["S"]
    if case["op"] == "evict":
        lens = _spread(case["low"], case["high"], S)
        n = -(-max(1, case["high"]) // 16) * 16
        # live tokens' scores, the maps read and written
        return dict(bytes=4 * (sum(lens) * case["live"] + 2 * S * n + S * case["freed"] + 3 * S), flops=0)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    new, lens = zip(*_sessions(case))
    T = sum(new)
    live = [m + (n - m) * case["live"] for m, n in zip(new, lens)]
    pairs = sum(m * (k - m) + m * (m + 1) // 2 for m, k in zip(new, live))
    ids = 4 * sum(lens) if case["maps"] else 4 * sum(lens) / case["page"]
    if case["op"] == "attend":
        return dict(bytes=4 * sum(live) * Hkv * D + ids + 4 * T * Hq * D + 4 * T * Hq, flops=4 * pairs * Hq * D)
    n = max(lens) if case["maps"] else -(-max(lens) // case["page"]) * case["page"]
    return dict(bytes=2 * sum(live) * Hkv * D + ids + 2 * T * Hq * D + 4 * T * Hq + 8 * S * n, flops=2 * pairs * Hq * D)


# ---------------------------------------------------------------------------
# the operators' definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_parts(st, s):
    """For each kv head of session s: (head, live positions, their slots, logits in 64 bits [rows][live], seen)."""
    case = st["case"]
    Hkv, G, page = case["Hkv"], case["Hq"] // case["Hkv"], case["page"]
    n, a, b = st["lens_host"][s], st["cu_host"][s], st["cu_host"][s + 1]
    pos = torch.arange(n, device=DEVICE)
    if st["slots"] is not None:
        pos = pos[(st["slots"][s, :n] != st["dead"]) & (st["slots"][s, :n] >= 0)]
        slot = st["slots"][s].long()[pos]
    else:
        slot = st["table"][s].long().repeat_interleave(page)[:n] * page + pos % page
    at = torch.arange(n - (b - a), n, device=DEVICE).repeat_interleave(G)
    for h in range(Hkv):
        q = st["q"][a:b, h * G:(h + 1) * G].double().reshape(-1, case["D"])
        x = q @ st["k_pool"][slot // page, slot % page, h].double().T * st["scale"]
        yield h, pos, slot, x, pos[None] <= at[:, None]


def _exact_attend(st):
    case = st["case"]
    T, Hq, D, page, G = st["cu_host"][-1], case["Hq"], case["D"], case["page"], case["Hq"] // case["Hkv"]
    out = torch.empty((T, Hq, D), dtype=torch.float64, device=DEVICE)
    lse = torch.empty((T, Hq), dtype=torch.float64, device=DEVICE)
    for s in range(case["S"]):
        a, b = st["cu_host"][s], st["cu_host"][s + 1]
        for h, _, slot, x, seen in _exact_parts(st, s):
            x[~seen] = -math.inf
            total = torch.logsumexp(x, 1)
            p = torch.exp(x - torch.where(torch.isinf(total), 0.0, total)[:, None])
            o = p @ st["v_pool"][slot // page, slot % page, h].double()
            out[a:b, h * G:(h + 1) * G] = o.view(b - a, G, D)
            lse[a:b, h * G:(h + 1) * G] = total.view(b - a, G)
    return dict(out=out, lse=lse)


def _exact_mass(st):
    case = st["case"]
    G = case["Hq"] // case["Hkv"]
    score = st["before"].double()
    for s in range(case["S"]):
        a, b = st["cu_host"][s], st["cu_host"][s + 1]
        for h, pos, _, x, seen in _exact_parts(st, s):
            lse = st["lse"][a:b, h * G:(h + 1) * G].double().reshape(-1, 1)
            p = torch.where(seen & torch.isfinite(lse), torch.exp(x - lse), 0.0)
            score[s, pos] += p.sum(0)
    return dict(score=score)


def exact(case, seed):
    if case["op"] == "evict":
        return None  # whole numbers only
    st = prepare(case, seed)
    return _exact_attend(st) if case["op"] == "attend" else _exact_mass(st)
