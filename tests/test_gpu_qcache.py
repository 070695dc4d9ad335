"""GPU parity of the 4-bit history cache against float64 numpy (qcache_ref):
stored codes and parameters bit for bit, attention over cached rows and the
weights they receive within bounds derived from the arithmetic, eviction row
for row, and the operators run one behind the other as a server runs them.

Everything outside the rows of a call is filled with patterns that would show:
codes and parameters of all ones (a NaN scale), NaN activations, NaN outputs."""
import numpy as np
import pytest
import torch

from hstu_pointwise_attention_b200 import ops

import qcache_ref as R
from gpu_common import assert_close

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
# The error of P beyond its logit's (R.attend): a part of P's size and a part of
# |x|.  CUDA cores: the exponential, the quotient and the logit's scaling, a few
# roundings each.  Tensor cores: P rounded to bf16, and SiLU(x) = h (1 + tanh h),
# h = x / 2, with a tanh whose relative error is at most 2^-10.98, which moves P
# by |h| 2^-10.98; the weights come from P ahead of its rounding, by an
# exponential and a quotient good to 2^-22 each.
U_CUDA = (16 * R.F32_U, 0.0)
U_TENSOR = (R.BF16_U + 2.0 ** -20, 2.0 ** -11.9)
U_W = (2.0 ** -20, 0.0)


def tensor_cores(p, impl):
    return p.dtype == "bf16" and impl == "auto" and p.dk == p.dv and p.dk in (64, 128)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def poisoned(rows, H, dk, dv):
    c = ops.QuantCache.empty(rows, H, dk, dv)
    for n in ("k_codes", "v_codes"):
        getattr(c, n).fill_(255)
    for n in ("k_scales", "v_scales"):
        getattr(c, n).fill_(-1)
    c.times.fill_(-(2 ** 62))
    c.pos.fill_(2 ** 31 - 1)
    c.weight.fill_(float("nan"))
    return c


def act(rng, shape, dtype):
    x = rng.standard_normal(shape)
    x = x / (1 + np.exp(-x))
    return torch.from_numpy(x.astype(np.float32)).cuda().to(DT[dtype])


def strided(t, pad, shift=0):
    """The same values in a buffer with wider rows, NaN around them."""
    T, H, d = t.shape
    buf = torch.full((T * (H * d + pad) + shift,), float("nan"), dtype=t.dtype, device=t.device)
    v = torch.as_strided(buf, (T, H, d), (H * d + pad, d, 1), shift)
    v.copy_(t)
    return v


def stored(c, rows, n):
    sl = slice(int(rows), int(rows) + int(n))
    cpu = lambda t: t[:, sl].cpu().numpy()
    return (R.unpack(cpu(c.k_codes), cpu(c.k_scales)), R.unpack(cpu(c.v_codes), cpu(c.v_scales)))


# ---------------------------------------------------------------------------
# Append and read
# ---------------------------------------------------------------------------
def hard_values(rng, shape):
    """Groups at which the format can go wrong."""
    T, H, d = shape
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-8, 8, (T, H, 1)))
    kinds = [lambda g: 0 * g, lambda g: -np.abs(g), lambda g: np.abs(g) + 100,
             lambda g: np.where(np.arange(32) == 3, 5.0, 0.0),            # one value
             lambda g: (np.arange(32) - 7) * 0.5,                          # ties of the rounding
             lambda g: np.arange(32) % 16 * 1.0,                           # span of exactly 15
             lambda g: np.where(np.arange(32) % 2, 7.5, -7.5),            # both ends round up
             lambda g: g * 1e-39, lambda g: g * 1e37,                      # subnormal, huge
             lambda g: np.where(np.arange(32) == 0, np.nan, g),
             lambda g: np.where(np.arange(32) == 1, np.inf, g),
             lambda g: np.where(np.arange(32) == 2, -np.inf, np.nan)]
    for t in range(T):
        g = x[t].reshape(-1, 32)
        for i in range(len(g)):
            if (t + i) % 3 == 0:
                g[i] = kinds[(t // 3 + i) % len(kinds)](g[i])
    return x


@pytest.mark.parametrize("H,dk,dv", [(1, 32, 32), (2, 64, 64), (8, 128, 128), (3, 96, 256),
                                     (2, 256, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_stores_the_defined_codes(H, dk, dv, dtype):
    rng = np.random.default_rng(100 + dk + H)
    lens, rows = [37, 0, 1, 18], [40, 3, 9, 11]
    off = np.concatenate([[0], np.cumsum(lens)])
    T = int(off[-1])
    with np.errstate(over="ignore", invalid="ignore"):
        k, v = (torch.from_numpy(hard_values(rng, (T, H, d)).astype(np.float32)).cuda()
                .to(DT[dtype]) for d in (dk, dv))
    ts = torch.arange(T, device="cuda") * 7 + 10 ** 12
    c, before = poisoned(80, H, dk, dv), poisoned(80, H, dk, dv)
    # whole rows aligned, wider rows, and rows that start off any 16-byte boundary
    for pad, shift in [(0, 0), (8, 0), (3, 1)]:
        for t in ("k_codes", "k_scales", "v_codes", "v_scales", "times", "pos", "weight"):
            getattr(c, t).copy_(getattr(before, t))
        ops.qcache_append(c, strided(k, pad, shift), strided(v, pad, shift), ts, off, rows,
                          [5, 6, 7, 2 ** 31 - 18])
        torch.cuda.synchronize()
        touched = torch.zeros(80, dtype=torch.bool, device="cuda")
        for b, n in enumerate(lens):
            sl = slice(rows[b], rows[b] + n)
            touched[sl] = True
            for x, cn, sn in ((k, "k_codes", "k_scales"), (v, "v_codes", "v_scales")):
                codes, params = R.pack(*R.quantise(f64(x[off[b]:off[b + 1]])))
                np.testing.assert_array_equal(getattr(c, cn)[:, sl].cpu().numpy(), codes)
                np.testing.assert_array_equal(
                    getattr(c, sn)[:, sl].cpu().numpy().view(np.uint16), params)
            assert torch.equal(c.times[sl], ts[off[b]:off[b + 1]])
            first = [5, 6, 7, 2 ** 31 - 18][b]
            assert c.pos[sl].tolist() == list(range(first, first + n))
            assert torch.all(c.weight[sl] == 0)
        for t in ("k_codes", "k_scales", "v_codes", "v_scales"):
            assert torch.equal(getattr(c, t)[:, ~touched], getattr(before, t)[:, ~touched])
        assert torch.equal(c.times[~touched], before.times[~touched])
        assert torch.all(c.weight[~touched].isnan())
    # and back: exact in both types, into wide and unaligned rows too
    for dt in ("bf16", "f32"):
        for pad, shift in [(0, 0), (8, 0), (1, 1)]:
            ko = strided(torch.zeros(T, H, dk, dtype=DT[dt], device="cuda"), pad, shift)
            vo = strided(torch.zeros(T, H, dv, dtype=DT[dt], device="cuda"), pad, shift)
            ops.qcache_read(c, rows, lens, k=ko, v=vo)
            for b, n in enumerate(lens):
                rk, rv = stored(c, rows[b], n)
                np.testing.assert_array_equal(f64(ko[off[b]:off[b + 1]]), rk)
                np.testing.assert_array_equal(f64(vo[off[b]:off[b + 1]]), rv)


def test_append_and_read_many_sequences():
    rng = np.random.default_rng(110)
    B = 150                                    # several launches' tables
    lens = rng.integers(0, 5, B)
    off = np.concatenate([[0], np.cumsum(lens)])
    order = rng.permutation(B)                 # regions in any order
    rows = np.zeros(B, np.int64)
    rows[order] = np.concatenate([[0], np.cumsum(lens[order] + 1)[:-1]])
    T, R_ = int(off[-1]), int((lens + 1).sum())
    k = act(rng, (T, 2, 64), "bf16")
    c = poisoned(R_, 2, 64, 64)
    ops.qcache_append(c, k, k, torch.arange(T, device="cuda"), off, rows, np.arange(B))
    ko, vo = ops.qcache_read(c, rows, lens)
    want = R.values(*R.quantise(f64(k)))
    np.testing.assert_array_equal(f64(ko), want)
    np.testing.assert_array_equal(f64(vo), want)
    assert c.times[torch.from_numpy(np.repeat(rows - off[:-1], lens) + np.arange(T)).cuda()
                   ].tolist() == list(range(T))


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
class Problem:
    """Sequences of cached rows and candidates, on the device and in float64."""

    def __init__(self, lens, cands, H, dk, dv, dtype, seed, nb=(40, 24), sub=2, per_head=False,
                 t_step=600, t_cand=None, alpha=None, shift=0, pad=0):
        rng = np.random.default_rng(seed)
        self.lens, self.n = np.array(lens), np.array(cands)
        B = len(lens)
        cap = self.lens + rng.integers(1, 6, B)
        self.rows = np.concatenate([[0], np.cumsum(cap)[:-1]]) + 1
        self.off = np.concatenate([[0], np.cumsum(self.n)])
        T, total = int(self.off[-1]), int(cap.sum()) + 1
        self.c = poisoned(total, H, dk, dv)
        self.dtype, self.H, self.dk, self.dv = dtype, H, dk, dv
        self.pos, self.cand_pos = [], []
        for b in range(B):
            L = int(lens[b])
            if L:
                sl = slice(int(self.rows[b]), int(self.rows[b]) + L)
                ops.qcache_append(self.c, act(rng, (L, H, dk), "bf16"),
                                  act(rng, (L, H, dv), "bf16") - 0.2,
                                  torch.zeros(L, dtype=torch.int64, device="cuda"), [0, L],
                                  [self.rows[b]], [0])
                # gaps in the positions, and rows in no order, as evictions leave them
                pos = np.sort(rng.choice(4 * L, L, replace=False))
                t = 10 ** 9 + np.cumsum(rng.integers(1, 2 * t_step, L))
                order = rng.permutation(L)
                self.c.pos[sl] = torch.from_numpy(pos[order].astype(np.int32)).cuda()
                self.c.times[sl] = torch.from_numpy(t[order]).cuda()
                self.c.weight[sl] = torch.from_numpy(rng.random(L).astype(np.float32)).cuda()
            self.cand_pos.append(4 * L)
        self.cand_pos = np.array(self.cand_pos)
        end = [int(self.c.times[self.rows[b]:self.rows[b] + lens[b]].max()) if lens[b] else 10 ** 9
               for b in range(B)]
        t = np.repeat(end, self.n) + 500
        if t_cand == "apart":          # every candidate its own time
            t = t + 977 * np.arange(T)
        elif t_cand == "before":       # earlier than part of the history
            t = t - rng.integers(0, 40 * t_step, T)
        self.t = t.astype(np.int64)
        self.ts = torch.from_numpy(self.t).cuda()
        q, k, v = act(rng, (T, H, dk), dtype), act(rng, (T, H, dk), dtype), act(rng, (T, H, dv), dtype)
        self.q, self.k, self.v = (strided(x, pad, shift) if pad or shift else x for x in (q, k, v))
        tab = lambda m: (rng.standard_normal((H, m) if per_head else m) * 0.5).astype(np.float32)
        self.rab_p, self.rab_t = tab(nb[0]), tab(nb[1])
        self.per_head, self.sub = per_head, sub
        self.alpha = 1 / np.sqrt(dk) if alpha is None else alpha
        self.scale = 1.0 / max(1, int((self.lens + self.n).max()))
        self.msl = int((self.lens + self.n).max())

    def run(self, decay=None, out=None, **kw):
        out = torch.full((int(self.off[-1]) + 2, self.H, self.dv), float("nan"),
                         dtype=DT[self.dtype], device="cuda") if out is None else out
        kw = {**dict(out=out, weight_decay=decay), **kw}
        return ops.attn_fwd_candidates_qcache(
            self.q, self.k, self.v, self.c, self.rows, self.lens, self.off, self.cand_pos, self.ts,
            torch.from_numpy(self.rab_p).cuda(), torch.from_numpy(self.rab_t).cuda(),
            max_seq_len=self.msl, time_bucket_sub_bits=self.sub, alpha=self.alpha,
            silu_scale=self.scale, rab_per_head=self.per_head, **kw)

    def reference(self, u):
        q, k, v = f64(self.q), f64(self.k), f64(self.v)
        for b in range(len(self.lens)):
            sl = slice(int(self.rows[b]), int(self.rows[b] + self.lens[b]))
            kh, vh = stored(self.c, self.rows[b], self.lens[b])
            a = slice(int(self.off[b]), int(self.off[b + 1]))
            yield b, sl, a, R.attend(q[a], k[a], v[a], kh, vh, self.c.pos[sl].cpu().numpy(),
                                     self.c.times[sl].cpu().numpy(), int(self.cand_pos[b]),
                                     self.t[a], self.rab_p, self.rab_t, self.sub, self.alpha,
                                     self.scale, *u)


def check(p, decay=0.75, impl="auto", **kw):
    """Output and weights against float64, and nothing else written."""
    before = p.c.weight.clone()
    T = int(p.off[-1])
    out = p.run(decay, impl=impl, **kw)
    torch.cuda.synchronize()
    got, w = f64(out), f64(p.c.weight)
    u_out = R.BF16_U if p.dtype == "bf16" else R.F32_U
    touched = np.zeros(len(w), bool)
    refs = []
    for (b, sl, a, (ref, bound, _, _)), (_, _, _, (_, _, step, wb)) in zip(
            p.reference(U_TENSOR if tensor_cores(p, impl) else U_CUDA),
            p.reference(U_W)):
        err = np.abs(got[a] - ref)
        assert np.all(err <= bound + u_out * (np.abs(ref) + bound)), \
            (b, float((err - bound - u_out * np.abs(ref)).max()))
        refs.append(ref)
        if decay is not None:
            want = decay * f64(before)[sl] + step if decay else step
            assert np.all(np.abs(w[sl] - want) <= wb + 2 * R.F32_U * (np.abs(want) + wb)), b
            touched[sl] = True
    if p.dtype == "bf16" and T and sum(r.size for r in refs) >= 256:
        assert_close(got[:T], np.concatenate(refs), "bf16", "attention over the 4-bit cache")
    assert np.all(np.isnan(got[T:])), "rows behind the last candidate were written"
    np.testing.assert_array_equal(w[~touched], f64(before)[~touched])
    return out[:T]


EDGES = dict(lens=[0, 1, 127, 128, 129, 300, 5, 64], cands=[3, 1, 17, 0, 64, 65, 130, 16])


@pytest.mark.parametrize("dtype,impl", [("bf16", "auto"), ("bf16", "simt"), ("f32", "auto")])
@pytest.mark.parametrize("H,dk,dv", [(2, 128, 128), (2, 64, 64), (1, 32, 96), (3, 256, 64)])
def test_attention_edges(dtype, impl, H, dk, dv):
    check(Problem(**EDGES, H=H, dk=dk, dv=dv, dtype=dtype, seed=200 + dk), impl=impl)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(t_cand="apart"), dict(t_cand="before"),
                                dict(t_cand="apart", t_step=10 ** 6), dict(t_step=10 ** 11),
                                dict(t_cand="apart", sub=0), dict(t_cand="apart", sub=8),
                                dict(per_head=True), dict(nb=(1, 1)), dict(nb=(1000, 1000), sub=4),
                                dict(nb=(5000, 3000), sub=8, t_cand="before"),
                                dict(pad=8), dict(pad=5, shift=1), dict(alpha=0.0),
                                dict(alpha=-3.0)], ids=str)
def test_attention_variants(dtype, kw):
    check(Problem([260, 33], [20, 70], 2, 128, 128, dtype, seed=230, **kw))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 2, 8, 31, 63, 64, 127, 128, 129, 200])
def test_attention_candidate_counts(dtype, n):
    check(Problem([200], [n], 2, 64, 64, dtype, seed=240 + n))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(per_head=True, t_cand="apart"),
                                dict(t_cand="before", sub=8, nb=(5000, 3000)),
                                dict(t_step=10 ** 11, t_cand="apart", pad=8),
                                dict(pad=5, shift=1, nb=(1, 1)), dict(alpha=-3.0)], ids=str)
def test_attention_few_candidates(d, kw):
    """Up to 8 candidates per sequence: histories that end at, before and behind
    the 32 keys of a step and the 128 of a tile, and ones split over CTAs."""
    check(Problem([0, 1, 31, 32, 33, 127, 128, 129, 160, 1000, 0, 3],
                  [1, 2, 3, 4, 5, 6, 7, 8, 1, 3, 8, 0], 2, d, d, "bf16", seed=240 + d, **kw))


def test_attention_few_candidates_hidden_buckets_and_one_more():
    p = Problem([150, 150, 40], [5, 8, 2], 2, 128, 128, "bf16", seed=248, t_cand="apart")
    p.rab_p[10:] = float("-inf")
    p.rab_t[5:12] = float(torch.finfo(torch.float32).min)
    check(p)
    p.rab_p[:] = float("-inf")
    out = p.run(0.0)
    assert torch.all(out[:int(p.off[-1])].float() == 0)
    for b in range(3):
        assert torch.all(p.c.weight[p.rows[b]:p.rows[b] + p.lens[b]] == 0)
    check(Problem([150, 150, 40], [5, 9, 2], 2, 128, 128, "bf16", seed=249))


def test_attention_calls_on_two_streams_at_once():
    """Each call has its own workspace: neither disturbs the other."""
    ps = [Problem([3000, 700], n, 2, 128, 128, "bf16", seed=256 + n[0])
          for n in ([1, 8], [70, 20], [200, 3])]
    want, weights = [], []
    for p in ps:
        w0 = p.c.weight.clone()
        want.append(p.run(0.5).clone())
        weights.append(p.c.weight.clone())
        p.c.weight.copy_(w0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    outs = [torch.full_like(w, float("nan")) for w in want]
    torch.cuda.synchronize()
    for p, s, o in zip(ps, streams, outs):
        p.run(0.5, out=o, stream=s)
    torch.cuda.synchronize()
    for p, o, w, cw in zip(ps, outs, want, weights):
        n = int(p.off[-1])
        assert torch.equal(o[:n], w[:n])
        assert torch.equal(p.c.weight.view(torch.int32), cw.view(torch.int32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_split_over_keys_and_many_sequences(dtype):
    check(Problem([5000], [1], 1, 128, 128, dtype, seed=250))          # one row, many ranges
    check(Problem([2000, 700], [129, 40], 2, 64, 64, dtype, seed=251))
    rng = np.random.default_rng(252)
    check(Problem(rng.integers(0, 40, 130), rng.integers(0, 4, 130), 2, 64, 64, dtype, seed=253))
    check(Problem([900] * 70, [70] * 70, 4, 128, 128, dtype, seed=254))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("low", [float("-inf"), float(torch.finfo(torch.float32).min), -1e31])
def test_attention_bias_that_hides_buckets(dtype, low):
    """Position and time buckets of -inf or the lowest float leave nothing of
    their rows, also where both tables say so and where no row is left."""
    p = Problem([150, 150, 40], [5, 70, 2], 2, 128, 128, dtype, seed=260)
    p.rab_p[10:] = low
    p.rab_t[5:12] = low
    check(p)
    p.rab_p[:] = low
    p.rab_t[:] = low
    out = p.run(0.0)
    assert torch.all(out[:int(p.off[-1])].float() == 0)
    for b in range(3):
        assert torch.all(p.c.weight[p.rows[b]:p.rows[b] + p.lens[b]] == 0)


def test_attention_weights_are_optional_and_decay():
    p = Problem([300, 10], [7, 0], 2, 64, 64, "bf16", seed=270)
    w0 = p.c.weight.clone()
    a = p.run(None)
    assert torch.equal(p.c.weight.view(torch.int32), w0.view(torch.int32))
    b = check(p, 0.0)
    # the weights' SiLU is computed more exactly; outputs agree to their rounding
    torch.testing.assert_close(a[:7].float(), b.float(), rtol=2 ** -6, atol=1e-3)
    check(p, 1.0)
    p.c.weight[p.rows[1]:p.rows[1] + 10] = float("nan")      # decay 0 does not read the old one
    p.run(0.0)
    assert torch.all(p.c.weight[p.rows[1]:p.rows[1] + 10] == 0)


def test_attention_overlapping_regions_and_no_cache():
    p = Problem([300, 200], [4, 9], 2, 64, 64, "bf16", seed=280)
    p.rows[1], p.cand_pos[1] = p.rows[0] + 20, p.cand_pos[0]        # a shared history
    check(p, None)
    with pytest.raises(ops.HstuError):
        p.run(1.0)
    e = Problem([0, 0], [3, 1], 2, 64, 64, "bf16", seed=281)
    e.c = ops.QuantCache.empty(0, 2, 64, 64)
    e.rows[:] = 0
    check(e, None)
    n = Problem([20], [0], 2, 64, 64, "bf16", seed=282)
    check(n, 0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_is_the_same_every_time_and_in_a_graph(dtype):
    p = Problem([3000, 100, 0], [70, 3, 2], 2, 128, 128, dtype, seed=290)
    w0 = p.c.weight.clone()
    first, w1 = p.run(0.5).clone(), None
    w1 = p.c.weight.clone()
    rp, rt = torch.from_numpy(p.rab_p).cuda(), torch.from_numpy(p.rab_t).cuda()
    out = torch.full_like(first, float("nan"))
    call = lambda: ops.attn_fwd_candidates_qcache(
        p.q, p.k, p.v, p.c, p.rows, p.lens, p.off, p.cand_pos, p.ts, rp, rt, max_seq_len=p.msl,
        time_bucket_sub_bits=p.sub, alpha=p.alpha, silu_scale=p.scale, weight_decay=0.5, out=out)
    same = lambda a, b: torch.equal(a.view(torch.int16 if a.dtype == DT["bf16"] else torch.int32),
                                    b.view(torch.int16 if b.dtype == DT["bf16"] else torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    p.c.weight.copy_(w0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()                              # another stream, eager
    torch.cuda.synchronize()
    T = int(p.off[-1])
    assert same(out[:T], first[:T]) and same(p.c.weight, w1)
    with torch.cuda.stream(side):
        with torch.cuda.graph(g):
            call()
    for _ in range(2):
        out.fill_(float("nan"))
        p.c.weight.copy_(w0)
        g.replay()
        torch.cuda.synchronize()
        assert same(out[:T], first[:T]) and same(p.c.weight, w1)
    p.c.weight.copy_(w0)                    # a stream given to the call
    torch.cuda.synchronize()
    ops.attn_fwd_candidates_qcache(
        p.q, p.k, p.v, p.c, p.rows, p.lens, p.off, p.cand_pos, p.ts, rp, rt, max_seq_len=p.msl,
        time_bucket_sub_bits=p.sub, alpha=p.alpha, silu_scale=p.scale, weight_decay=0.5, out=out,
        stream=side)
    torch.cuda.synchronize()
    assert same(out[:T], first[:T]) and same(p.c.weight, w1)


def test_attention_row_offsets_past_32_bits():
    """Rows behind the first 2^32 bytes of codes of one cache."""
    rows = 2 ** 32 // 64 // 2 + 4096            # H = 2, d = 128: 64 bytes of codes per row
    p = Problem([300], [5], 2, 128, 128, "bf16", seed=295)
    big = ops.QuantCache(*(torch.empty((2, rows, w), dtype=t, device="cuda") for w, t in
                           ((64, torch.uint8), (4, torch.int16), (64, torch.uint8),
                            (4, torch.int16))),
                         *(torch.empty(rows, dtype=t, device="cuda") for t in
                           (torch.int64, torch.int32, torch.float32)))
    at, to = slice(int(p.rows[0]), int(p.rows[0]) + 300), slice(rows - 301, rows - 1)
    for n in ("k_codes", "k_scales", "v_codes", "v_scales"):
        getattr(big, n)[:, to] = getattr(p.c, n)[:, at]
    for n in ("times", "pos", "weight"):
        getattr(big, n)[to] = getattr(p.c, n)[at]
    want, w = p.run(0.5), None
    w = p.c.weight[at].clone()
    p.c, p.rows = big, np.array([rows - 301])
    got = p.run(0.5)
    assert torch.equal(got[:5], want[:5]) and torch.equal(big.weight[to], w)
    k, v = ops.qcache_read(big, p.rows, [300])
    n = ops.qcache_evict(big, p.rows, [300], [100], [2 ** 31 - 1])
    assert n.tolist() == [100]
    src = R.evict(f64(w), np.zeros(300), 100, 1)
    k2, v2 = ops.qcache_read(big, p.rows, n)
    assert torch.equal(k2, k[src]) and torch.equal(v2, v[src])


# ---------------------------------------------------------------------------
# Eviction
# ---------------------------------------------------------------------------
NAMES = ("k_codes", "k_scales", "v_codes", "v_scales", "times", "pos", "weight")


def random_cache(rng, lens, H, dk, dv, ties=True):
    cap = np.asarray(lens) + rng.integers(1, 4, len(lens))
    rows = np.concatenate([[0], np.cumsum(cap)[:-1]])
    n = int(cap.sum())
    g = lambda hi, shape, dt: torch.from_numpy(rng.integers(0, hi, shape)).to(dt).cuda()
    w = rng.standard_normal(n).astype(np.float32)
    if ties:
        w = (np.round(w * 4) / 4).astype(np.float32)      # -0.0 and 0.0 among them
        w[rng.random(n) < 0.05] = np.nan
        w[rng.random(n) < 0.05] = np.inf
        w[rng.random(n) < 0.05] = -np.inf
    pos = np.concatenate([rng.permutation(c) for c in cap]).astype(np.int32)
    return rows, ops.QuantCache(
        g(256, (H, n, dk // 2), torch.uint8), g(2 ** 15, (H, n, dk // 32), torch.int16),
        g(256, (H, n, dv // 2), torch.uint8), g(2 ** 15, (H, n, dv // 32), torch.int16),
        g(2 ** 60, n, torch.int64), torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda())


def copy_of(c):
    return ops.QuantCache(*(getattr(c, n).clone() for n in NAMES))


def same_rows(a, ra, b, rb):
    for n in NAMES:
        x, y = getattr(a, n), getattr(b, n)
        if n == "weight":
            x, y = x.view(torch.int32), y.view(torch.int32)
        x, y = (x[:, ra], y[:, rb]) if x.dim() == 3 else (x[ra], y[rb])
        assert torch.equal(x, y), n


def check_evict(lens, budgets, keep_pos, H=2, dk=64, dv=64, seed=300, ties=True):
    rng = np.random.default_rng(seed)
    rows, c = random_cache(rng, lens, H, dk, dv, ties)
    old = copy_of(c)
    w, pos = c.weight.cpu().numpy(), c.pos.cpu().numpy()
    n = np.minimum(lens, budgets)
    srcs = [R.evict(w[r:r + L], pos[r:r + L], k, kp)
            for r, L, k, kp in zip(rows, lens, budgets, keep_pos)]
    # into another cache, at other rows
    to = np.concatenate([[0], np.cumsum(n + 2)[:-1]]) + 1
    dst = copy_of(random_cache(rng, [int((n + 2).sum()) + 2], H, dk, dv)[1])
    dst_old = copy_of(dst)
    got = ops.qcache_evict(c, rows, lens, budgets, keep_pos, dst=dst, dst_rows=to)
    assert got.tolist() == n.tolist()
    everything = slice(0, c.rows)
    same_rows(c, everything, old, everything)                 # the source is only read
    rest = torch.ones(dst.rows, dtype=torch.bool, device="cuda")
    for b, s in enumerate(srcs):
        i = torch.tensor(s, dtype=torch.int64, device="cuda") + int(rows[b])
        j = torch.arange(len(s), device="cuda") + int(to[b])
        same_rows(dst, j, old, i)
        rest[j] = False
    same_rows(dst, rest, dst_old, rest)
    # in place: rows behind the kept ones are left as they were
    ops.qcache_evict(c, rows, lens, budgets, keep_pos)
    rest = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    for b, s in enumerate(srcs):
        i = torch.tensor(s, dtype=torch.int64, device="cuda") + int(rows[b])
        j = torch.arange(len(s), device="cuda") + int(rows[b])
        same_rows(c, j, old, i)
        rest[j] = False
    same_rows(c, rest, old, rest)


@pytest.mark.parametrize("ties", [True, False])
@pytest.mark.parametrize("H,dk,dv", [(2, 64, 64), (1, 32, 256), (8, 128, 128)])
def test_evict_edges(H, dk, dv, ties):
    lens = [0, 1, 1, 5, 31, 33, 1023, 1024, 1025, 3001, 100, 100, 100]
    keep = [4, 0, 1, 3, 31, 2, 1022, 500, 1, 2000, 100, 400, 50]
    kp = [0, 0, 0, 2 ** 31 - 1, 0, 30, 1000, 900, 1020, -5, 10, 10, 0]
    check_evict(lens, keep, kp, H, dk, dv, ties=ties)


def test_evict_many_sequences_and_long_ones():
    rng = np.random.default_rng(310)
    lens = rng.integers(0, 60, 140)
    check_evict(lens, rng.integers(0, 60, 140), rng.integers(0, 80, 140), seed=311)
    # longer than the keys that fit in shared memory, beside a short one
    check_evict([50001, 17], [30000, 9], [49990, 3], 1, 32, 32, seed=312)


def test_evict_graph_replay_trims_again():
    rng = np.random.default_rng(320)
    rows, c = random_cache(rng, [400, 77], 2, 64, 64)
    start = copy_of(c)
    args = (rows, [400, 77], [100, 50], [390, 70])
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    ops.qcache_evict(c, *args, workspace=ws)
    want = copy_of(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g):
            ops.qcache_evict(c, *args, workspace=ws)
    torch.cuda.synchronize()
    for n in NAMES:
        getattr(c, n).copy_(getattr(start, n))
    g.replay()
    torch.cuda.synchronize()
    same_rows(c, slice(0, c.rows), want, slice(0, c.rows))


# ---------------------------------------------------------------------------
# The layer, and the operators one behind the other
# ---------------------------------------------------------------------------
def layer_params(rng, H, d, D):
    F, n1 = H * d, 4 * H * d
    w = lambda *s: (rng.standard_normal(s) / np.sqrt(s[1])).astype(np.float32)
    b = lambda n: (0.1 * rng.standard_normal(n)).astype(np.float32)
    bf = lambda x: torch.from_numpy(x).cuda().to(torch.bfloat16)
    f = lambda x: torch.from_numpy(x).cuda()
    return (bf(w(n1, D)), f(b(n1)), f(1 + b(F)), f(b(F)), bf(w(D, F)), f(b(D)), f(b(40)), f(b(24)))


def layer_ref(x, P, c, rows, lens, off, cpos, ct, H, d, sub, scale, residual, proj):
    """float64 layer from the projection that the kernel stored (its rounding
    of U, V, Q, K is the layer's own)."""
    w1, b1, ga, be, w2, b2, rp, rt = (f64(t) for t in P)
    F = H * d
    z = x @ w1.T + b1
    exact = z / (1 + np.exp(-z))
    assert_close(proj, exact, "bf16", "projection")
    u, v, q, k = (proj[:, i * F:(i + 1) * F] for i in range(4))
    a = np.zeros((len(x), F))
    steps = []
    for b in range(len(lens)):
        sl, m = slice(int(rows[b]), int(rows[b] + lens[b])), slice(int(off[b]), int(off[b + 1]))
        kh, vh = stored(c, rows[b], lens[b])
        o, _, step, _ = R.attend(*(t[m].reshape(-1, H, d) for t in (q, k, v)), kh, vh,
                                 c.pos[sl].cpu().numpy(), c.times[sl].cpu().numpy(), int(cpos[b]),
                                 ct[m], rp, rt, sub, 1 / np.sqrt(d), scale, 0.0)
        a[m] = o.reshape(-1, F)
        steps.append((sl, step))
    mu = a.mean(1, keepdims=True)
    g = (a - mu) / np.sqrt(((a - mu) ** 2).mean(1, keepdims=True) + 1e-5) * ga + be
    return (x if residual else 0) + (g * u) @ w2.T + b2, steps


@pytest.mark.parametrize("H,d,D,residual", [(2, 128, 64, True), (4, 64, 256, False),
                                            (1, 32, 40, True), (8, 128, 512, True)])
def test_layer_over_the_cache(H, d, D, residual):
    rng = np.random.default_rng(400 + d + H)
    p = Problem([260, 0, 70], [33, 2, 1], H, d, d, "bf16", seed=401)
    P = layer_params(rng, H, d, D)
    x = torch.from_numpy(rng.standard_normal((36, D)).astype(np.float32)).cuda().bfloat16()
    proj = torch.full((36, 4 * H * d), float("nan"), dtype=torch.bfloat16, device="cuda")
    before = p.c.weight.clone()
    kw = dict(num_heads=H, d_qk=d, d_v=d, max_seq_len=p.msl, time_bucket_sub_bits=2,
              silu_scale=p.scale, residual=residual)
    y = ops.layer_fwd_candidates_qcache(x, *P, p.c, p.rows, p.lens, p.off, p.cand_pos, p.ts,
                                        weight_decay=0.5, proj_out=proj, **kw)
    ref, steps = layer_ref(f64(x), P, p.c, p.rows, p.lens, p.off, p.cand_pos, p.t, H, d, 2,
                           p.scale, residual, f64(proj))
    assert_close(f64(y), ref, "bf16", "layer over the 4-bit cache")
    for sl, step in steps:
        want = 0.5 * f64(before)[sl] + step
        np.testing.assert_allclose(f64(p.c.weight)[sl], want, rtol=1e-4, atol=1e-7)
    # without the optional outputs: the same rows
    y2 = ops.layer_fwd_candidates_qcache(x, *P, p.c, p.rows, p.lens, p.off, p.cand_pos, p.ts, **kw)
    assert_close(f64(y2), ref, "bf16", "layer, no weights")
    empty = ops.layer_fwd_candidates_qcache(x[:0], *P, p.c, p.rows, p.lens, [0, 0, 0, 0],
                                            p.cand_pos, p.ts[:0], weight_decay=0.25, **kw)
    assert empty.shape == (0, D)


def test_serving_loop_append_attend_evict():
    """History pass -> cache -> candidates -> a new event -> eviction -> the
    next candidates, two users, one layer, as a server runs it."""
    H, d, D, sub, scale = 2, 64, 128, 2, 1 / 256
    rng = np.random.default_rng(420)
    P = layer_params(rng, H, d, D)
    hist, budget, F = [130, 61], [100, 100], H * d
    off = np.array([0, 130, 191])
    x = torch.from_numpy(rng.standard_normal((191, D)).astype(np.float32)).cuda().bfloat16()
    t = np.concatenate([10 ** 9 + np.cumsum(rng.integers(1, 900, n)) for n in hist])
    ts = torch.from_numpy(t).cuda()
    kw = dict(num_heads=H, d_qk=d, d_v=d, max_seq_len=256, time_bucket_sub_bits=sub,
              silu_scale=scale)
    _, proj = ops.layer_fwd_keep_proj(x, *P, off, ts, **kw)
    rows = np.array([0, 200])
    c = poisoned(400, H, d, d)
    # the cache is filled from the projection's columns in place (strided rows)
    ops.qcache_append(c, proj[:, 3 * F:], proj[:, F:2 * F], ts, off, rows, [0, 0])
    kq, vq = ops.qcache_read(c, rows, hist)
    np.testing.assert_array_equal(
        f64(kq), R.values(*R.quantise(f64(proj[:, 3 * F:]).reshape(-1, H, d))))
    lens, pos_next = np.array(hist), np.array(hist)
    w = [np.zeros(130), np.zeros(61)]
    for step in range(3):
        coff = np.array([0, 5, 5 + 3])
        xc = torch.from_numpy(rng.standard_normal((8, D)).astype(np.float32)).cuda().bfloat16()
        ct = np.repeat([t[129], t[190]], [5, 3]) + 1000 * (step + 1)
        cts = torch.from_numpy(ct).cuda()
        pc = torch.empty((8, 4 * F), dtype=torch.bfloat16, device="cuda")
        y = ops.layer_fwd_candidates_qcache(xc, *P, c, rows, lens, coff, pos_next, cts,
                                            weight_decay=0.9, proj_out=pc, **kw)
        ref, steps = layer_ref(f64(xc), P, c, rows, lens, coff, pos_next, ct, H, d, sub, scale,
                               True, f64(pc))
        assert_close(f64(y), ref, "bf16", f"candidates, step {step}")
        for b, (sl, s) in enumerate(steps):
            w[b] = 0.9 * w[b] + s
            np.testing.assert_allclose(f64(c.weight)[sl], w[b], rtol=1e-4, atol=1e-7)
        # the first candidate of each user becomes an event
        pick = torch.tensor([0, 5], device="cuda")
        ev = pc[pick]
        ops.qcache_append(c, ev[:, 3 * F:], ev[:, F:2 * F], cts[pick], [0, 1, 2], rows + lens,
                          pos_next)
        lens, pos_next = lens + 1, pos_next + 1
        w = [np.append(a, 0.0) for a in w]
        # trim; the last 10 positions stay
        cw, cp = c.weight.cpu().numpy(), c.pos.cpu().numpy()
        srcs = [R.evict(cw[r:r + n], cp[r:r + n], k, q) for r, n, k, q in
                zip(rows, lens, budget, pos_next - 10)]
        old = copy_of(c)
        new = ops.qcache_evict(c, rows, lens, budget, pos_next - 10)
        for b, s in enumerate(srcs):
            i = torch.tensor(s, device="cuda") + int(rows[b])
            same_rows(c, slice(int(rows[b]), int(rows[b]) + len(s)), old, i)
            w[b] = w[b][s]
            kept = cp[rows[b]:rows[b] + lens[b]][s]
            assert set(range(int(pos_next[b]) - 10, int(pos_next[b]))) <= set(kept.tolist())
        lens = new
        assert lens.tolist() == [min(a, 100) for a in (130 + 1 if step == 0 else 101, 62 + step)]
