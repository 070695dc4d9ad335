"""Cases for the 4-bit key / value cache of the M-FALCON candidate path.

Four operators, reached through hstu_pointwise_attention_b200.ops:
  append  quantise new tokens' keys and values into the cache (qcache_append),
          read back as the values they stand for (qcache_read)
  attend  candidates (or one new event) against the cached history
          (attn_fwd_candidates_qcache), optionally adding up how much weight each
          cached row received
  evict   keep a user's `budget` most used rows (qcache_evict), read back
  layer   a whole HSTU layer on candidate rows over the cache
          (layer_fwd_candidates_qcache)

The 4-bit format: groups of 32 values along the head dimension share a scale
s (a float with 4 significant bits) and a zero point z in 0..15; a value is
s (q - z), q in 0..15.  Eight codes make a 32-bit word: nibble i holds element
2 i, nibble i + 4 element 2 i + 1 (i = 0..3).  A group's parameter is 16 bits:
the upper 12 bits of s as a bfloat16, then z.
"""
import math
import random

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SLACK = 17          # rows of a user's region behind its last token
TS_START = 1_700_000_000


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _case(op, users, heads, d, hist, new, dtype="bf16", nb=128, sub_bits=2, per_head=False,
          weights=False, same_time=True, keep=0.0, d_model=0, name=None):
    c = {"op": op, "users": users, "heads": heads, "d": d, "hist_lo": hist[0], "hist_hi": hist[1],
         "new_lo": new[0], "new_hi": new[1], "dtype": dtype, "nb": nb, "sub_bits": sub_bits,
         "per_head": per_head, "weights": weights, "same_time": same_time, "keep": keep,
         "d_model": d_model}
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new event of each of 8 active users enters the cache: latency
        _case("append", 8, 8, 128, (0, 0), (1, 1), name="append_8x1"),
        # the history pass of the M-FALCON workload fills the cache: bandwidth
        _case("append", 8, 8, 128, (0, 0), (4096, 4096), name="append_8x4096"),
        # 32 users with ragged histories, 4 heads of 64, float32 activations
        _case("append", 32, 4, 64, (0, 0), (64, 1024), dtype="f32", name="append_32_ragged_f32"),
        # one user's next event against a 4096-token history: the smallest attention call
        _case("attend", 1, 8, 128, (4096, 4096), (1, 1), name="attend_1x1"),
        # one event of each of 64 users with heavy-tailed histories up to 8192: cache bandwidth
        _case("attend", 64, 8, 128, (512, 8192), (1, 1), nb=256, sub_bits=3, weights=True,
              name="attend_64x1_ragged_w"),
        # an M-FALCON micro-batch: 8 users x 256 candidates, weights kept for eviction
        _case("attend", 8, 8, 128, (4096, 4096), (256, 256), weights=True,
              name="attend_8x256_w"),
        # long histories, all candidates in one call, each with its own time: tensor cores
        _case("attend", 4, 8, 128, (8192, 8192), (1024, 1024), nb=256, sub_bits=3,
              same_time=False, name="attend_4x1024"),
        # 32 ragged users, 4 heads of 64, float32, tables per head: a few candidates each
        _case("attend", 32, 4, 64, (64, 1024), (1, 24), dtype="f32", per_head=True, weights=True,
              name="attend_32_ragged_f32_w"),
        # one user's cache trimmed after a burst of events: latency of the selection
        _case("evict", 1, 8, 128, (4096, 4096), (0, 0), keep=0.9375, name="evict_1x4096"),
        # 32 users' ragged histories halved: selection and bandwidth
        _case("evict", 32, 8, 128, (1024, 8192), (0, 0), keep=0.5, name="evict_32_ragged"),
        # one event of each of 8 users through a whole layer
        _case("layer", 8, 8, 128, (4096, 4096), (1, 1), d_model=512, name="layer_8x1"),
        # an M-FALCON micro-batch through a whole layer
        _case("layer", 8, 8, 128, (4096, 4096), (256, 256), d_model=512, name="layer_8x256"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "evict", "layer"])
    users, heads = _log(rng, 1, 64), rng.choice([2, 4, 8])
    d = rng.choice([64, 128])
    dtype = "bf16" if op == "layer" else rng.choice(["bf16", "bf16", "bf16", "f32"])
    nb, sub_bits = rng.choice([(32, 0), (128, 2), (256, 3)])
    if op == "append":
        hi = _log(rng, 1, min(4096, 32768 // users))
        return _case(op, users, heads, d, (0, 0), (max(1, hi // 3), hi), dtype=dtype)
    hi = _log(rng, 16, min(8192, 65536 // users))
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    if op == "evict":
        return _case(op, users, heads, d, (lo, hi), (0, 0), dtype=dtype,
                     keep=rng.choice([0.25, 0.5, 0.75, 0.96875]))
    top = 1024 if dtype == "bf16" else 48
    n = _log(rng, 1, max(1, min(top, 8192 * 4096 // (users * hi))))
    heads = 2 ** rng.randrange(1, 4)
    return _case(op, users, heads, d, (lo, hi), (max(1, n // 2), n), dtype=dtype, nb=nb,
                 sub_bits=sub_bits, per_head=op == "attend" and rng.random() < 0.5,
                 weights=op == "attend" and rng.random() < 0.6, same_time=rng.random() < 0.7,
                 d_model=rng.choice([256, 512]) if op == "layer" else 0)


def _lens(case):
    """Users' history and new-token counts: a part of the case, not of the inputs."""
    r = random.Random(7 * case["users"] + case["hist_hi"] + 3 * case["new_hi"])
    pick = lambda lo, hi: 0 if hi == 0 else _log(r, lo, hi)  # noqa: E731
    hist = [pick(case["hist_lo"], case["hist_hi"]) for _ in range(case["users"])]
    new = [pick(case["new_lo"], case["new_hi"]) for _ in range(case["users"])]
    return np.array(hist, np.int64), np.array(new, np.int64)


def _offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


def _budget(case, hist):
    return np.maximum(1, np.floor(hist * case["keep"])).astype(np.int64)


# ---------------------------------------------------------------------------
# The 4-bit format (plain form)
# ---------------------------------------------------------------------------
def _quantise(x):
    """x [T, H, d] -> codes uint8 [H, T, d / 2], params int16 [H, T, d / 32]."""
    T, H, d = x.shape
    g = x.double().reshape(T, H, d // 32, 32).nan_to_num(nan=0.0).clamp(-2.0 ** 126, 2.0 ** 126)
    lo, hi = g.amin(-1).clamp(max=0.0), g.amax(-1).clamp(min=0.0)
    # the smallest s of 4 significant bits with 15 s >= hi - lo
    m, e = torch.frexp((hi - lo) / 15.0)
    s = torch.ldexp(torch.ceil(m * 16.0), e - 4).clamp(min=2.0 ** -126)
    z = torch.round(-lo / s)
    q = (torch.round(g / s[..., None]) + z[..., None]).clamp(0, 15)
    s = torch.where(hi > lo, s, 0.0)
    z = torch.where(hi > lo, z, 0.0).to(torch.int32)
    q = torch.where((hi > lo)[..., None], q, 0.0).to(torch.int32)
    params = ((s.float().view(torch.int32) >> 16) | z).to(torch.int16)
    q = q.reshape(T, H, d // 8, 4, 2)
    at = torch.arange(4, device=x.device, dtype=torch.int32) * 4
    w = ((q[..., 0] << at) | (q[..., 1] << (at + 16))).sum(-1).to(torch.int32)
    return (w.transpose(0, 1).contiguous().view(torch.uint8),
            params.transpose(0, 1).contiguous())


def _values(codes, params):
    """The float32 values [H, R, d] that codes and params stand for."""
    H, R, half = codes.shape
    w = codes.view(torch.int32)
    at = torch.arange(4, device=codes.device, dtype=torch.int32) * 4
    q = torch.stack([(w[..., None] >> at) & 15, (w[..., None] >> (at + 16)) & 15], -1)
    p = params.to(torch.int32)
    s = ((p & 0xFFF0) << 16).view(torch.float32)
    q = q.reshape(H, R, half // 16, 32) - (p & 15)[..., None]
    return (q.float() * s[..., None]).reshape(H, R, 2 * half)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) + 1)
    return g


def _act(g, shape, dtype):
    """Activations as the layer's projection gives them: SiLU of a normal."""
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.sigmoid(x)).to(dtype)


def _events(g, n):
    """n increasing event times, gaps of 600 s on the mean."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return TS_START + torch.cumsum((-600.0 * torch.log1p(-u)).round().clamp(min=1).long(), 0)


def prepare(case, seed):
    g, dt = _gen(seed), DT[case["dtype"]]
    H, d = case["heads"], case["d"]
    hist, new = _lens(case)
    cap = hist + SLACK + (new if case["op"] == "append" else 0)
    rows = _offsets(cap)
    R = int(rows[-1])
    rows = rows[:-1].copy()
    off = _offsets(new)
    T = int(off[-1])
    s = {"case": dict(case), "rows": rows, "hist": hist, "off": off, "dtype": dt, "R": R}
    if case["op"] == "append":
        s["k"], s["v"] = _act(g, (T, H, d), dt), _act(g, (T, H, d), dt)
        s["ts"] = _events(g, T)
        s["pos"] = np.arange(case["users"], dtype=np.int32) * 3
        s["cache"] = _empty_cache(R, H, d)
        return s
    # a cache in use: rows of every user, positions with gaps where rows were evicted before
    kc, ks = _quantise(_act(g, (R, H, d), torch.bfloat16))
    vc, vs = _quantise(_act(g, (R, H, d), torch.bfloat16))
    step = np.random.RandomState(seed % (2 ** 31)).randint(0, 10, R)
    pos = np.cumsum(1 + 3 * (step == 0)).astype(np.int64)
    pos -= np.repeat(pos[rows], cap)
    times = _events(g, R)
    weight = torch.rand(R, generator=g, device="cuda")
    weight = (weight * 64).floor() / 64 if case["op"] == "evict" else weight  # equal ones among them
    s["cache"] = {"k_codes": kc, "k_scales": ks, "v_codes": vc, "v_scales": vs, "times": times,
                  "pos": torch.from_numpy(pos.astype(np.int32)).cuda(), "weight": weight}
    last = rows + np.maximum(hist - 1, 0)
    s["cand_pos"] = (pos[last] + 1).astype(np.int32)
    if case["op"] == "evict":
        s["budget"] = _budget(case, hist)
        s["keep_pos"] = (s["cand_pos"] - np.minimum(64, np.maximum(hist // 8, 1))).astype(np.int32)
        s["dst_rows"] = _offsets(s["budget"] + SLACK)
        s["dst"] = _empty_cache(int(s["dst_rows"][-1]), H, d)
        s["dst_rows"] = s["dst_rows"][:-1].copy()
        return s
    user = torch.from_numpy(np.repeat(np.arange(case["users"]), new)).cuda()
    at = torch.arange(T, device="cuda")
    s["cand_ts"] = times[torch.from_numpy(last).cuda()][user] + 700
    if not case["same_time"]:
        s["cand_ts"] = s["cand_ts"] + 40 * (at - torch.from_numpy(off).cuda()[user])
    s["weight0"] = weight.clone()
    tab = (H, case["nb"]) if case["per_head"] else (case["nb"],)
    s["rab_p"] = 0.02 * torch.randn(tab, generator=g, device="cuda")
    s["rab_t"] = 0.02 * torch.randn(tab, generator=g, device="cuda")
    msl = int(case["hist_hi"] + case["new_hi"])
    s["msl"], s["alpha"], s["scale"] = msl, 1.0 / math.sqrt(d), 1.0 / msl
    if case["op"] == "attend":
        s["q"], s["k"], s["v"] = (_act(g, (T, H, d), dt) for _ in range(3))
        return s
    D, F, n1 = case["d_model"], H * d, 4 * H * d
    uni = lambda *sh: ((2 * torch.rand(sh, generator=g, device="cuda") - 1) *  # noqa: E731
                       math.sqrt(6.0 / (sh[0] + sh[1]))).to(torch.bfloat16)
    s["x"] = torch.randn((T, D), generator=g, device="cuda").to(torch.bfloat16)
    s["w1"], s["w2"] = uni(n1, D), uni(D, F)
    s["b1"] = 0.1 * torch.randn(n1, generator=g, device="cuda")
    s["b2"] = 0.1 * torch.randn(D, generator=g, device="cuda")
    s["gamma"] = 1 + 0.1 * torch.randn(F, generator=g, device="cuda")
    s["beta"] = 0.1 * torch.randn(F, generator=g, device="cuda")
    return s


def _empty_cache(R, H, d):
    z = lambda sh, t: torch.zeros(sh, dtype=t, device="cuda")  # noqa: E731
    return {"k_codes": z((H, R, d // 2), torch.uint8), "k_scales": z((H, R, d // 32), torch.int16),
            "v_codes": z((H, R, d // 2), torch.uint8), "v_scales": z((H, R, d // 32), torch.int16),
            "times": z(R, torch.int64), "pos": z(R, torch.int32), "weight": z(R, torch.float32)}


def _rows_of(rows, lens):
    """Global row of every token of every user, on the device."""
    off = _offsets(lens)
    at = np.arange(int(off[-1])) + np.repeat(rows - off[:-1], lens)
    return torch.from_numpy(at).cuda()


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    return {"append": _plain_append, "attend": _plain_attend, "evict": _plain_evict,
            "layer": _plain_layer}[case["op"]](s, case)


def _run_own(s, case):
    from hstu_pointwise_attention_b200 import ops
    if "handle" not in s:
        s["handle"] = ops.QuantCache(**s["cache"])
        if "dst" in s:
            s["dst_handle"] = ops.QuantCache(**s["dst"])
    cache, off = s["handle"], s["off"]
    if case["op"] == "append":
        ops.qcache_append(cache, s["k"], s["v"], s["ts"], off, s["rows"], s["pos"])
        k, v = ops.qcache_read(cache, s["rows"], np.diff(off), dtype=s["dtype"])
        return k, v, cache.times, cache.pos
    if case["op"] == "evict":
        dst = s["dst_handle"]
        ops.qcache_evict(cache, s["rows"], s["hist"], s["budget"], s["keep_pos"], dst=dst,
                      dst_rows=s["dst_rows"])
        k, v = ops.qcache_read(dst, s["dst_rows"], s["budget"], dtype=s["dtype"])
        return k, v, dst.times, dst.pos, dst.weight
    kw = dict(max_seq_len=s["msl"], time_bucket_sub_bits=case["sub_bits"], alpha=s["alpha"],
              silu_scale=s["scale"])
    if case["op"] == "layer":
        return ops.layer_fwd_candidates_qcache(
            s["x"], s["w1"], s["b1"], s["gamma"], s["beta"], s["w2"], s["b2"], s["rab_p"],
            s["rab_t"], cache, s["rows"], s["hist"], off, s["cand_pos"], s["cand_ts"],
            num_heads=case["heads"], d_qk=case["d"], d_v=case["d"], **kw)
    if case["weights"]:
        cache.weight.copy_(s["weight0"])
    out = ops.attn_fwd_candidates_qcache(
        s["q"], s["k"], s["v"], cache, s["rows"], s["hist"], off, s["cand_pos"], s["cand_ts"],
        s["rab_p"], s["rab_t"], rab_per_head=case["per_head"],
        weight_decay=0.5 if case["weights"] else None, **kw)
    return (out, cache.weight) if case["weights"] else out


def _plain_append(s, case):
    c, lens = s["cache"], np.diff(s["off"])
    at = _rows_of(s["rows"], lens)
    for n in ("k", "v"):
        codes, params = _quantise(s[n])
        c[n + "_codes"][:, at], c[n + "_scales"][:, at] = codes, params
    c["times"][at] = s["ts"]
    c["pos"][at] = torch.from_numpy(
        (np.arange(len(at)) + np.repeat(s["pos"] - s["off"][:-1], lens)).astype(np.int32)).cuda()
    c["weight"][at] = 0.0
    k, v = (_values(c[n + "_codes"][:, at], c[n + "_scales"][:, at]).transpose(0, 1) for n in "kv")
    return k.to(s["dtype"]), v.to(s["dtype"]), c["times"], c["pos"]


def _time_bucket(dt, sub, nb):
    e = torch.frexp(dt.clamp(min=1).double())[1].long() - 1
    up = (e - sub).clamp(min=0)
    b = torch.where(dt < 2 ** sub, dt.clamp(min=0),
                    (e - sub + 1) * 2 ** sub + (dt >> up) - 2 ** sub)
    return b.clamp(max=nb - 1)


def _attend(s, case, q, k, v):
    """float32 outputs [T, H, d] of the candidates, and the step's weights [R]."""
    c, off, hist = s["cache"], s["off"], s["hist"]
    new = np.diff(off)
    B, n, L = case["users"], int(new.max()), max(1, int(hist.max()))
    dev = q.device
    # users side by side, padded to the longest: rows [B, L], candidates [B, n]
    j, i = torch.arange(L, device=dev), torch.arange(n, device=dev)
    rows, hl = torch.from_numpy(s["rows"]).to(dev), torch.from_numpy(hist).to(dev)
    o, nl = torch.from_numpy(off[:-1].copy()).to(dev), torch.from_numpy(new).to(dev)
    at = rows[:, None] + torch.minimum(j[None], (hl[:, None] - 1).clamp(min=0))
    ct = o[:, None] + torch.minimum(i[None], (nl[:, None] - 1).clamp(min=0))
    seen = (j[None] < hl[:, None])[:, None, :] & (i[None] < nl[:, None])[:, :, None]
    kh = _values(c["k_codes"], c["k_scales"])[:, at]          # [H, B, L, d]
    vh = _values(c["v_codes"], c["v_scales"])[:, at]
    qc = q[ct].permute(2, 0, 1, 3)                            # [H, B, n, d]
    x = s["alpha"] * (qc @ kh.transpose(-1, -2))
    dp = (torch.from_numpy(s["cand_pos"]).to(dev).long()[:, None] - c["pos"][at]).clamp(0, case["nb"] - 1)
    bt = _time_bucket(s["cand_ts"][ct][:, :, None] - c["times"][at][:, None, :],
                      case["sub_bits"], case["nb"])
    rp, rt = s["rab_p"].reshape(-1, case["nb"]), s["rab_t"].reshape(-1, case["nb"])
    x = x + rp[:, dp][:, :, None, :] + rt[:, bt]
    p = torch.where(seen[None], x * torch.sigmoid(x), 0.0)
    user = torch.from_numpy(np.repeat(np.arange(B), new)).to(dev)
    seat = torch.arange(len(user), device=dev) - o[user]
    out = (p @ vh).permute(1, 2, 0, 3)[user, seat]
    x = s["alpha"] * (q * k).sum(-1) + rp[:, 0] + rt[:, 0]
    out = s["scale"] * (out + (x * torch.sigmoid(x))[..., None] * v)
    step = torch.zeros(s["R"], device=dev)
    mine = j[None] < hl[:, None]
    step[at[mine]] = s["scale"] * p.abs().sum((0, 2))[mine]
    return out, step, at[mine]


def _plain_attend(s, case):
    out, step, at = _attend(s, case, s["q"].float(), s["k"].float(), s["v"].float())
    out = out.to(s["dtype"])
    if not case["weights"]:
        return out
    w = s["weight0"].clone()
    w[at] = 0.5 * w[at] + step[at]
    return out, w


def _plain_evict(s, case):
    c, hist, keep = s["cache"], s["hist"], s["budget"]
    B, L = case["users"], int(hist.max())
    dev = c["times"].device
    j = torch.arange(L, device=dev)[None]
    rows, hl, kl, kp = (torch.from_numpy(np.asarray(a, np.int64)).to(dev)[:, None]
                        for a in (s["rows"], hist, keep, s["keep_pos"]))
    at = rows + torch.minimum(j, hl - 1)
    key = c["weight"][at].nan_to_num(nan=-math.inf)
    key = torch.where(c["pos"][at] >= kp, math.inf, key)
    key = torch.where(j < hl, key, -math.inf)
    order = torch.argsort(key, dim=1, descending=True, stable=True)
    kept = torch.zeros((B, L), dtype=torch.bool, device=dev)
    kept.scatter_(1, order, j.expand(B, L) < kl)
    src = torch.arange(L, device=dev).repeat(B, 1)
    # kept rows behind the budget fill the holes before it, both in order
    src[~kept & (j < kl)] = j.expand(B, L)[kept & (j >= kl)]
    src = (rows + src)[j.expand(B, L) < kl]
    to = _rows_of(s["dst_rows"], keep)
    d = s["dst"]
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        d[n][:, to] = c[n][:, src]
    for n in ("times", "pos", "weight"):
        d[n][to] = c[n][src]
    k, v = (_values(d[n + "_codes"][:, to], d[n + "_scales"][:, to]).transpose(0, 1) for n in "kv")
    return k.to(s["dtype"]), v.to(s["dtype"]), d["times"], d["pos"], d["weight"]


def _plain_layer(s, case):
    H, d = case["heads"], case["d"]
    F = H * d
    x = s["x"].float()
    z = x @ s["w1"].float().t() + s["b1"]
    z = z * torch.sigmoid(z)
    u, v, q, k = z.split(F, dim=1)
    a, _, _ = _attend(s, case, *(t.reshape(-1, H, d) for t in (q, k, v)))
    a = a.reshape(-1, F)
    a = a - a.mean(1, keepdim=True)
    a = a * torch.rsqrt(a.square().mean(1, keepdim=True) + 1e-5) * s["gamma"] + s["beta"]
    return (x + (a * u) @ s["w2"].float().t() + s["b2"]).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# What one pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    H, d = case["heads"], case["d"]
    es = 2 if case["dtype"] == "bf16" else 4
    hist, new = _lens(case)
    Th, T = int(hist.sum()), int(new.sum())
    row4 = 2 * H * (d // 2 + 2 * (d // 32))        # K and V of one row, 4-bit
    row = 2 * H * d * es                           # and as activations
    if case["op"] == "append":
        return {"bytes": T * (row + 8 + row4 + 16 + row), "flops": 0}
    if case["op"] == "evict":
        n = int(_budget(case, hist).sum())
        return {"bytes": 8 * Th + n * (2 * row4 + 32 + row), "flops": 0}
    tabs = 8 * case["nb"] * (H if case["per_head"] else 1)
    w = {"bytes": Th * (row4 + 12 + (8 if case["weights"] else 0)) + T * (2 * row + 8) + tabs,
         "flops": 4 * d * H * int((new * (hist + 1)).sum())}
    if case["op"] == "layer":
        D, F = case["d_model"], H * d
        w["bytes"] = Th * (row4 + 12) + 2 * 5 * F * D + 4 * (6 * F + D) + T * (4 * D + 8) + tabs
        w["flops"] += 2 * T * 5 * F * D
    return w


# ---------------------------------------------------------------------------
# The definition in 64 bits, user by user
# ---------------------------------------------------------------------------
def _exact_code(x):
    """Values [T, H, d] after the 4-bit format, from its definition."""
    T, H, d = x.shape
    g = x.double().reshape(-1, 32)
    lo = torch.minimum(g.min(1).values, torch.zeros((), dtype=torch.float64, device=x.device))
    hi = torch.maximum(g.max(1).values, torch.zeros((), dtype=torch.float64, device=x.device))
    span = hi - lo
    e = torch.floor(torch.log2((span / 15).clamp(min=2.0 ** -126)))
    s = torch.full_like(span, math.inf)
    for de in (-1, 0, 1):                          # every scale near span / 15, the smallest that will do
        for m in range(8, 16):
            t = m / 8 * torch.exp2(e + de)
            s = torch.where((15 * t >= span) & (t < s) & (t >= 2.0 ** -126), t, s)
    z = torch.round(-lo / s)
    q = torch.clamp(torch.round(g / s[:, None]) + z[:, None], 0, 15)
    return torch.where(span[:, None] > 0, s[:, None] * (q - z[:, None]), 0.0).reshape(T, H, d)


def _exact_rows(codes, params):
    """Values [R, H, d] of cache rows, nibble by nibble."""
    b = codes.cpu().numpy().reshape(codes.shape[0], codes.shape[1], -1, 4)
    nib = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:3], 8)      # nibble 0..7 of each word
    q = nib[..., [0, 4, 1, 5, 2, 6, 3, 7]].reshape(*b.shape[:2], -1)
    p = params.cpu().numpy().astype(np.int64) & 0xFFFF
    s = ((p & 0xFFF0) << 16).astype(np.uint32).view(np.float32).astype(np.float64)
    x = (q.astype(np.float64) - np.repeat(p & 15, 32, axis=2)) * np.repeat(s, 32, axis=2)
    return torch.from_numpy(x).transpose(0, 1).cuda()


def _exact_attend(s, case, q, k, v):
    c, off = s["cache"], s["off"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    w = s["weight0"].double()
    rp = s["rab_p"].double().reshape(-1, case["nb"])
    rt = s["rab_t"].double().reshape(-1, case["nb"])
    silu = lambda x: x / (1 + torch.exp(-x))  # noqa: E731
    for b in range(case["users"]):
        r0, L = int(s["rows"][b]), int(s["hist"][b])
        a0, a1 = int(off[b]), int(off[b + 1])
        sl = slice(r0, r0 + L)
        kb = _exact_rows(c["k_codes"][:, sl], c["k_scales"][:, sl])
        vb = _exact_rows(c["v_codes"][:, sl], c["v_scales"][:, sl])
        dp = torch.clamp(int(s["cand_pos"][b]) - c["pos"][sl].long(), 0, case["nb"] - 1)
        dt = (s["cand_ts"][a0:a1, None] - c["times"][None, sl]).cpu().numpy()
        e = np.frexp(np.maximum(dt, 1).astype(np.float64))[1] - 1
        sub = case["sub_bits"]
        bt = np.where(dt <= 0, 0, np.where(dt < 2 ** sub, dt, (e - sub) * 2 ** sub +
                                           (np.maximum(dt, 0) >> np.maximum(e - sub, 0))))
        bt = torch.from_numpy(np.minimum(bt, case["nb"] - 1)).cuda()
        for h in range(case["heads"]):
            t = h if case["per_head"] else 0
            x = s["alpha"] * q[a0:a1, h] @ kb[:, h].t() + rp[t][dp][None] + rt[t][bt]
            p = silu(x)
            x = s["alpha"] * (q[a0:a1, h] * k[a0:a1, h]).sum(1) + rp[t][0] + rt[t][0]
            out[a0:a1, h] = s["scale"] * (p @ vb[:, h] + silu(x)[:, None] * v[a0:a1, h])
            w[sl] = (0.5 * w[sl] if h == 0 else w[sl]) + s["scale"] * p.abs().sum(0)
    return out, w


def exact(case, seed):
    s = prepare(case, seed)
    op, H, d = case["op"], case["heads"], case["d"]
    if op == "append":
        return _exact_code(s["k"]), _exact_code(s["v"]), None, None
    if op == "attend":
        out, w = _exact_attend(s, case, s["q"].double(), s["k"].double(), s["v"].double())
        return (out, w) if case["weights"] else out
    if op == "layer":
        F = H * d
        x = s["x"].double()
        z = x @ s["w1"].double().t() + s["b1"].double()
        z = z / (1 + torch.exp(-z))
        part = lambda i: z[:, i * F:(i + 1) * F].reshape(-1, H, d)  # noqa: E731
        a = _exact_attend(s, case, part(2), part(3), part(1))[0].reshape(-1, F)
        mean = a.sum(1, keepdim=True) / F
        a = (a - mean) / torch.sqrt(((a - mean) ** 2).sum(1, keepdim=True) / F + 1e-5)
        a = a * s["gamma"].double() + s["beta"].double()
        return x + (a * z[:, :F]) @ s["w2"].double().t() + s["b2"].double()
    # evict: sort every user's rows on the host
    c, ks, vs = s["cache"], [], []
    weight, pos = c["weight"].double().cpu().numpy(), c["pos"].cpu().numpy()
    w_out = torch.zeros(s["dst"]["weight"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["users"]):
        r0, L, n = int(s["rows"][b]), int(s["hist"][b]), int(s["budget"][b])
        score = [math.inf if pos[r0 + j] >= s["keep_pos"][b] else weight[r0 + j] for j in range(L)]
        kept = sorted(sorted(range(L), key=lambda j: (-score[j], j))[:n])
        tail = [j for j in kept if j >= n]
        stay = {j for j in kept if j < n}
        src = [j if j in stay else tail.pop(0) for j in range(n)]
        at = torch.tensor(src, device="cuda") + r0
        ks.append(_exact_rows(c["k_codes"][:, at], c["k_scales"][:, at]))
        vs.append(_exact_rows(c["v_codes"][:, at], c["v_scales"][:, at]))
        d0 = int(s["dst_rows"][b])
        w_out[d0:d0 + n] = c["weight"][at].double()
    return torch.cat(ks), torch.cat(vs), None, None, w_out
