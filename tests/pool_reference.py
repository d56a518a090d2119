"""Plain 64-bit implementations of the calls over the page pools (test infrastructure; shares nothing with the library):
attention through explicit lists of slots, the attention weight of every token, eviction by sorting.  With each value
comes the bound of a 32-bit evaluation's error that the tests hold the kernels to."""
import numpy as np
import torch

F64 = torch.float64


def sessions(cu, lens, T, reach):
    """(first row, rows, length) of each session, cut to what the arguments allow."""
    out = []
    for s, n in enumerate(lens):
        a, b = cu[s], cu[s + 1]
        count = 0 if a < 0 or b < a else max(0, min(b, T) - a)
        out.append((a, count, min(max(n, 0), reach)))
    return out


def _parts(q, k_pool, cu, lens, slots, live, scale, T=None):
    """For each session and kv head: rows of q, their live keys, logits, which are seen and each logit's error bound."""
    T = q.shape[0] if T is None else T
    Hkv, D, G = k_pool.shape[2], q.shape[2], q.shape[1] // k_pool.shape[2]
    k_flat = k_pool.flatten(0, 1)
    for s, (a, m, n) in enumerate(sessions(cu, lens, T, slots.shape[1])):
        if m == 0:
            continue
        pos = torch.nonzero(live[s, :n]).flatten()
        sl = slots[s, pos]
        at = torch.arange(n - m, n, device=q.device).repeat_interleave(G)
        for g in range(Hkv):
            rows = q[a:a + m, g * G:(g + 1) * G].to(F64).reshape(m * G, D)
            k = k_flat[sl, g].to(F64)
            x = scale * (rows @ k.T)
            # D products of two bf16 values and their sum, each step off by 2^-23 at most (the tensor cores cut off)
            delta = (D + 2) * 2.0 ** -23 * scale * (rows.abs() @ k.abs().T)
            yield s, a, m, g, G, pos, sl, x, pos[None] <= at[:, None], delta


def attend(q, k_pool, v_pool, cu, lens, slots, live, scale):
    """out, lse and their tolerances; rows of no session are NaN."""
    T, Hq, D = q.shape
    out, out_tol = (torch.full((T, Hq, D), float("nan"), dtype=F64, device=q.device) for _ in range(2))
    lse, lse_tol = (torch.full((T, Hq), float("nan"), dtype=F64, device=q.device) for _ in range(2))
    v_flat = v_pool.flatten(0, 1)
    for _, a, m, g, G, _, sl, x, seen, delta in _parts(q, k_pool, cu, lens, slots, live, scale):
        x = x.masked_fill(~seen, -torch.inf)
        total = torch.logsumexp(x, 1) if x.shape[1] else torch.full(x.shape[:1], -torch.inf, dtype=F64, device=q.device)
        empty = total == -torch.inf
        p = torch.exp(x - torch.where(empty, 0.0, total)[:, None])
        v = v_flat[sl, g].to(F64)
        o, mass = p @ v, p @ v.abs()
        d = torch.where(seen, delta, 0.0).amax(1) if x.shape[1] else torch.zeros_like(total)
        n = seen.sum(1)
        # weights are rounded to bf16 (2^-8), exp2 and the sums over n tokens take 2^-23 a step; the output rounds once more
        rel = 2.0 ** -8 + 2 * d + (n + 16) * 2.0 ** -23
        put = lambda t, y: t[a:a + m, g * G:(g + 1) * G].copy_(y.view(m, G, *y.shape[1:]))  # noqa: E731
        put(out, o), put(lse, total)
        put(out_tol, 2.0 ** -8 * o.abs() + rel[:, None] * mass * (1 + 2.0 ** -7) + 1e-30)
        put(lse_tol, d + (n + 16) * 2.0 ** -23 + 2.0 ** -22 * torch.where(empty, 0.0, total.abs()) + 1e-6)
    return out, lse, out_tol, lse_tol


def check_attend(got, got_lse, want):
    out, lse, out_tol, lse_tol = want
    rows = ~torch.isnan(lse)
    got, got_lse = got.to(F64), got_lse.to(F64)
    assert torch.equal(torch.isinf(got_lse)[rows], torch.isinf(lse)[rows]) and not torch.isnan(got_lse[rows]).any()
    fin = rows & ~torch.isinf(lse)
    off = (got_lse - lse).abs()[fin]
    assert (off <= lse_tol[fin]).all(), (off / lse_tol[fin]).max()
    off = (got - out).abs()[rows]
    assert (off <= out_tol[rows]).all(), (off / out_tol[rows]).max()
    assert not got[rows & torch.isinf(lse)].any()


def mass(q, lse, k_pool, cu, lens, slots, live, scale, before, T=None):
    """The score [S][reach] that before becomes, and its tolerance."""
    score = before.to(F64).clone()
    tol = torch.zeros_like(score)
    terms = torch.zeros_like(score)
    for s, a, m, g, G, pos, _, x, seen, delta in _parts(q, k_pool, cu, lens, slots, live, scale, T):
        l = lse[a:a + m, g * G:(g + 1) * G].to(F64).reshape(-1, 1)
        seen = seen & (l != -torch.inf)
        l = torch.where(l == -torch.inf, 0.0, l)
        p = torch.where(seen, torch.exp(x - l), 0.0)
        # the exponent: the logit's error, and x and lse scaled and subtracted in 32 bits; exp2 itself 2^-22
        e = delta + (x.abs() + l.abs()) * 2.0 ** -22 + 2.0 ** -21
        score[s, pos] += p.sum(0)
        tol[s, pos] += torch.where(seen, p * torch.expm1(e), 0.0).sum(0)
        terms[s, pos] += seen.sum(0)
    # fp32 sums of positive terms: each of the n steps off by 2^-24 of the sum; then the old score's
    return score, tol * (1 + 2.0 ** -10) + (terms + 64) * 2.0 ** -24 * score.abs() + 1e-30


def check_mass(got, want):
    score, tol = want
    off = (got.to(F64) - score).abs()
    assert (off <= tol).all(), (off / tol).max()


def evict(score, lens, budget, slots, dead, n_sink, n_recent, room=None):
    """numpy: slot maps, freed slots of each session and their counts, one session after the other by sorting."""
    score, slots = np.asarray(score, np.float32), np.array(slots)
    out, freed = slots.copy(), []
    for s, n in enumerate(lens):
        n = min(max(int(n), 0), slots.shape[1])
        live = [j for j in range(n) if slots[s, j] >= 0 and slots[s, j] != dead]
        may = [j for j in live if n_sink <= j < n - n_recent]
        count = max(0, min(len(live) - int(budget[s]), len(may), len(may) if room is None else room))
        rank = lambda j: (0, 0.0, -j) if np.isnan(score[s, j]) else (1, float(score[s, j]), -j)  # noqa: E731
        gone = sorted(sorted(may, key=rank)[:count])
        freed.append([int(slots[s, j]) for j in gone])
        out[s, gone] = dead
    return out, freed, [len(f) for f in freed]
