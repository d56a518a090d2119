"""Plain 64-bit implementations of the serving operators, on the CPU: the 4-bit cache format, slot planning and
attention with explicit masks (test infrastructure; shares nothing with the library)."""
import numpy as np
import torch

MAGS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def scale_value(byte):
    """Value of a scale byte: 5 exponent bits (bias 15), 3 mantissa bits; 255 is NaN."""
    b = np.asarray(byte, np.int64)
    e, m = b >> 3, b & 7
    v = np.where(e == 0, m * 2.0 ** -17, (1 + m / 8) * 2.0 ** (e - 15.0))
    return np.where(b == 255, np.nan, v)


LADDER = scale_value(np.arange(227))  # the scales in use: 0 .. 10240


def quantise(x):
    """[..., D] -> codes u8 [..., D/2], scale bytes u8 [..., D/16]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, 16)
    mag = np.abs(g)
    with np.errstate(invalid="ignore"):
        broken = ~(mag <= 61440).all(-1)
        top = np.where(broken, 0, mag.max(-1))
    byte = np.searchsorted(6 * LADDER, top)  # first scale with 6 s >= top (exact in 64 bits)
    s = np.where(byte > 0, LADDER[byte], 1.0)[..., None]
    y = np.where(broken[..., None], 0, mag) / s  # 53-bit quotient of a 24-bit by a 4-bit number: ties stay ties
    d = np.abs(y[..., None] - MAGS)
    near = d == d.min(-1, keepdims=True)
    code = np.where(near, np.array([0, 1, 0, 1, 0, 1, 0, 1]), 9).argmin(-1)  # of two nearest, the even one
    code = code + 8 * np.signbit(g)
    code = np.where(broken[..., None], 0, code).reshape(*x.shape)
    byte = np.where(broken, 255, byte)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), byte.astype(np.uint8)


def dequantise(codes, scales):
    codes = np.asarray(codes, np.int64)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(c & 8, -1.0, 1.0) * MAGS[c & 7]
    return v * np.repeat(scale_value(scales), 16, -1)


def attention(q, k, v, seen, scale):
    """q [R][D], k, v [N][D], seen [R][N] bool -> (out [R][D], lse [R], absolute weighted sum [R][D], logit error unit [R]):
    the last two bound rounding errors: sum p |v| / l, and the largest seen scale * sum |q||k|."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    out, mass = np.zeros((q.shape[0], v.shape[1])), np.zeros((q.shape[0], v.shape[1]))
    lse, unit = np.full(q.shape[0], -np.inf), np.zeros(q.shape[0])
    for r in range(q.shape[0]):
        j = np.flatnonzero(seen[r])
        if not j.size:
            continue
        x = scale * (k[j] @ q[r])
        m = x.max()
        p = np.exp(x - m)
        lse[r] = m + np.log(p.sum())
        p /= p.sum()
        out[r] = p @ v[j]
        mass[r] = p @ np.abs(v[j])
        unit[r] = (scale * (np.abs(k[j]) @ np.abs(q[r]))).max()
    return out, lse, mass, unit


def plan(cached, new_len, free, page, P, table, T, ld):
    """What kvsel_plan_slots documents, one session after the other (valid lengths)."""
    table = np.array(table)
    cu, slots, pos, taken = [0], [], [], 0
    maps = np.full((len(cached), ld), -1, np.int64)
    for s, (c, n) in enumerate(zip(cached, new_len)):
        have, need = -(-c // page), -(-(c + n) // page)
        for j in range(have, need):
            table[s, j] = free[taken] if taken < len(free) else -1
            taken += 1
        at = lambda p: -1 if not 0 <= table[s, p // page] < P else table[s, p // page] * page + p % page  # noqa: E731
        slots += [at(p) for p in range(c, c + n)]
        pos += list(range(c, c + n))
        for p in range(min(c + n, ld)):
            maps[s, p] = at(p)
        cu.append(cu[-1] + n)
    total = len(slots)
    slots += [-1] * (T - total)
    pos += [-1] * (T - total)
    return table, np.array(cu), np.array(slots[:T]), np.array(pos[:T]), maps, np.array([total, taken])


def f64(t):
    return t.detach().cpu().double().numpy()


def torch_u8(a, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)
