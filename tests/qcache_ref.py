"""The 4-bit history cache in float64 numpy, from its definition
(include/hstu.h): the number format, attention over cached rows with the
weights they receive, and eviction.  Used by the cache's tests only."""
import math

import numpy as np

F32_U = 2.0 ** -24      # half a step of float32, relative
BF16_U = 2.0 ** -8      # and of bfloat16


def quantise(x):
    """x [T, H, d] -> (q int [T, H, d], s float64 [T, H, d/32], z int)."""
    T, H, d = x.shape
    g = np.asarray(x, np.float64).reshape(T, H, d // 32, 32)
    g = np.clip(np.where(np.isnan(g), 0.0, g), -2.0 ** 126, 2.0 ** 126)
    lo, hi = np.minimum(g.min(-1), 0.0), np.maximum(g.max(-1), 0.0)
    m, e = np.frexp((hi - lo) / 15.0)
    s = np.maximum(np.ldexp(np.ceil(m * 16.0) / 16.0, e), 2.0 ** -126)
    z = np.rint(-lo / s)
    q = np.clip(np.rint(g / s[..., None]) + z[..., None], 0, 15)
    live = hi > lo
    return (np.where(live[..., None], q, 0).astype(np.int64).reshape(T, H, d),
            np.where(live, s, 0.0), np.where(live, z, 0).astype(np.int64))


def values(q, s, z):
    d = q.shape[-1]
    g = q.reshape(*q.shape[:-1], d // 32, 32) - z[..., None]
    return (g * s[..., None]).reshape(*q.shape[:-1], d)


def pack(q, s, z):
    """(codes uint8 [H, T, d/2], params uint16 [H, T, d/32]) as stored."""
    T, H, d = q.shape
    w = np.zeros((T, H, d // 8), np.uint64)
    e = q.reshape(T, H, d // 8, 8).astype(np.uint64)
    for i in range(8):
        w |= e[..., i] << np.uint64(4 * (i // 2) + 16 * (i % 2))
    codes = w.astype("<u4").transpose(1, 0, 2).copy().view(np.uint8)
    bits = s.astype(np.float32).view(np.uint32) >> 16
    return codes, (bits | z.astype(np.uint32)).astype(np.uint16).transpose(1, 0, 2).copy()


def unpack(codes, params):
    """values float64 [T, H, d] of stored bytes."""
    w = np.ascontiguousarray(codes).view("<u4").astype(np.int64)      # [H, T, d/8]
    q = np.stack([(w >> (4 * (i // 2) + 16 * (i % 2))) & 15 for i in range(8)], -1)
    H, T = w.shape[:2]
    p = params.view(np.uint16).astype(np.uint32)
    s = ((p & 0xFFF0) << 16).view(np.float32).astype(np.float64)
    z = (p & 15).astype(np.int64)
    return values(q.reshape(H, T, 2 * codes.shape[2]), s, z).transpose(1, 0, 2)


def time_bucket(dt, sub, nb):
    dt = np.asarray(dt, np.int64)
    e = np.array([max(int(x), 1).bit_length() - 1 for x in dt.reshape(-1)],
                 np.int64).reshape(dt.shape)
    up = np.maximum(e - sub, 0)
    b = (e - sub + 1) * 2 ** sub + (np.maximum(dt, 0) >> up) - 2 ** sub
    b = np.where(dt <= 0, 0, np.where(dt < 2 ** sub, dt, b))
    return np.minimum(b, nb - 1)


def silu(x):
    """x sigmoid(x), 0 in the limit -inf."""
    e = np.exp(-np.abs(x))
    sig = np.where(x >= 0, 1 / (1 + e), e / (1 + e))
    return np.where(np.isneginf(x), 0.0, np.where(np.isneginf(x), 0.0, x) * sig)


def attend(q, k, v, kh, vh, hist_pos, hist_t, cand_pos, cand_t, rab_p, rab_t, sub, alpha, scale,
           u_p, u_abs=0.0, u_x=F32_U):
    """One sequence: q, k, v [n, H, d], kh, vh [L, H, d] -> (out, weight step,
    and for both the largest error that arithmetic may leave).

    The bounds: a logit is off by u_x per product and addition of its sum, P by
    SiLU' <= 1.1 times that, by u_p of its own size (its rounding, and what the
    exponential and quotient leave) and by u_abs |x| (a sigmoid with an absolute
    error), each sum by 2 u per term (an
    accumulator may truncate)."""
    n, H, dq = q.shape
    L = kh.shape[0]
    rp, rt = np.atleast_2d(rab_p), np.atleast_2d(rab_t)
    rp, rt = (np.broadcast_to(t, (H, t.shape[1])).astype(np.float64) for t in (rp, rt))
    out, bound = np.zeros((n, H, vh.shape[2])), np.zeros((n, H, vh.shape[2]))
    w, wb = np.zeros(L), np.zeros(L)
    dp = np.clip(cand_pos - np.asarray(hist_pos, np.int64), 0, rp.shape[1] - 1)
    bt = time_bucket(np.asarray(cand_t)[:, None] - np.asarray(hist_t)[None], sub, rt.shape[1])
    for h in range(H):
        bias = rp[h][dp][None] + rt[h][bt]
        x = alpha * q[:, h] @ kh[:, h].T + bias
        p = silu(x)
        size = abs(alpha) * np.abs(q[:, h]) @ np.abs(kh[:, h]).T
        seen = bias >= -1e30
        dp_abs = np.where(seen, 1.1 * u_x * (2 * (dq + 4) * size + 4 * np.abs(np.where(seen, bias, 0))), 0)
        dp_abs = dp_abs + u_p * np.abs(p) + u_abs * np.abs(np.where(seen, x, 0)) + 1e-30
        xs = alpha * (q[:, h] * k[:, h]).sum(1) + rp[h][0] + rt[h][0]
        ps = silu(xs)
        dps = (1.1 * u_x * (2 * (dq + 4) * abs(alpha) * np.abs(q[:, h] * k[:, h]).sum(1) +
                            4 * np.abs(rp[h][0] + rt[h][0])) + u_p * np.abs(ps) +
               u_abs * np.abs(xs))
        va = np.abs(vh[:, h])
        out[:, h] = scale * (p @ vh[:, h] + ps[:, None] * v[:, h])
        tot = np.abs(p) @ va + np.abs(ps)[:, None] * np.abs(v[:, h])
        bound[:, h] = abs(scale) * (dp_abs @ va + dps[:, None] * np.abs(v[:, h]) +
                                    2 * F32_U * (L + 8) * tot)
        w += scale * np.abs(p).sum(0)
        wb += abs(scale) * (dp_abs.sum(0) + 2 * F32_U * (n * H + 8) * np.abs(p).sum(0))
    return out, bound, w, wb


def evict(weight, pos, budget, keep_pos):
    """The row every kept row comes from."""
    L = len(weight)
    n = min(L, int(budget))
    score = [math.inf if pos[j] >= keep_pos else
             (-math.inf if math.isnan(weight[j]) else float(weight[j])) for j in range(L)]
    kept = set(sorted(range(L), key=lambda j: (-score[j], j))[:n])
    tail = iter(sorted(j for j in kept if j >= n))
    return [j if j in kept else next(tail) for j in range(n)]
