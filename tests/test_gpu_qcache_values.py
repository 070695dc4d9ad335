"""The 4-bit history cache's attention where its values are not ordinary:
infinities and NaN in a candidate or in a bias table, each of them kept to the
rows and sums that the definition gives it to."""
import numpy as np
import pytest
import torch

from hstu_pointwise_attention_b200 import ops

import qcache_ref as R
from gpu_common import assert_close
from test_gpu_qcache import Problem, f64, layer_params, stored

pytestmark = pytest.mark.gpu


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def run(p, decay, w0, **kw):
    """(out, weight) of a call from weights w0."""
    p.c.weight.copy_(w0)
    out = p.run(decay, **kw)[:int(p.off[-1])].clone()
    return out, p.c.weight.clone()


# 8: warp-level products; 9, 64: 64-wide tiles; 65 to 200: 128-wide tiles, one and two
@pytest.mark.parametrize("n", [8, 9, 64, 65, 128, 200])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("decay", [0.5, None])
def test_a_candidates_own_value_stays_its_own(n, d, decay):
    """out_j takes v_i for j = i only: an infinity or a NaN in one candidate's v
    leaves every other candidate's bits, and its own other features', alone."""
    p = Problem([300, 0, 40], [n, min(n, 20), 3], 2, d, d, "bf16", seed=500 + n)
    w0 = p.c.weight.clone()
    clean, w_clean = run(p, decay, w0)
    for i in (0, n // 2, n - 1, n + 1):            # the last one: a sequence without a history
        for bad in (float("inf"), float("-inf"), float("nan")):
            kept = p.v.clone()
            p.v[i, 1, 5] = bad
            got, w = run(p, decay, w0)
            p.v.copy_(kept)
            assert not torch.isfinite(got[i, 1, 5])
            got[i, 1, 5] = clean[i, 1, 5]
            assert torch.equal(bits(got), bits(clean)), (i, bad)
            assert torch.equal(bits(w), bits(w_clean))


@pytest.mark.parametrize("n", [8, 9, 65])
@pytest.mark.parametrize("what", ["q", "k"])
def test_a_candidates_own_query_and_key_stay_its_own(n, what):
    p = Problem([300, 0], [n, 9], 2, 128, 128, "bf16", seed=520 + n)
    clean, _ = run(p, None, p.c.weight.clone())
    for i in (0, 1, n - 1, n + 2):
        x = getattr(p, what)
        kept = x.clone()
        x[i, 0, 7] = float("nan")
        got, _ = run(p, None, p.c.weight.clone())
        x.copy_(kept)
        assert torch.isnan(got[i, 0]).all()
        got[i, 0] = clean[i, 0]
        assert torch.equal(bits(got), bits(clean)), i


# The error of P beyond its logit's, by the kernel that takes the call: CUDA cores,
# a few float32 roundings; bf16 kernels, P rounded to bf16 ahead of its product,
# its exponential and quotient good to 2^-22 each.  The weights come from P ahead
# of its rounding.
U_P = {"simt": 16 * R.F32_U, "bf16": R.BF16_U + 2.0 ** -20}
U_W = {"simt": 16 * R.F32_U, "bf16": 2.0 ** -20}


def agree(got, ref, tol, what):
    """NaN where the definition has NaN, the same infinities, and the rest within tol."""
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref), err_msg=what)
    inf = np.isinf(ref)
    np.testing.assert_array_equal(got[inf], ref[inf], err_msg=what)
    fin = np.isfinite(ref)
    assert np.all(np.isfinite(got[fin])), what
    assert np.all(np.abs(got - ref)[fin] <= tol[fin]), \
        (what, float((np.abs(got - ref) - tol)[fin].max()))


def check_values(p, decay=0.75, impl="auto"):
    """Outputs and weights against float64, non-finite ones among them."""
    kind = "bf16" if p.dtype == "bf16" and impl == "auto" and p.dk == p.dv and \
        p.dk in (64, 128) else "simt"
    u_out = R.BF16_U if p.dtype == "bf16" else R.F32_U
    w0 = p.c.weight.clone()
    got, w = run(p, decay, w0, impl=impl)
    got, w, w0 = f64(got), f64(w), f64(w0)
    with np.errstate(invalid="ignore", over="ignore"):
        outs = [x[3][:2] + (x[2],) for x in p.reference((U_P[kind], 0.0))]
        steps = [x[3][2:] + (x[1],) for x in p.reference((U_W[kind], 0.0))]
        for (ref, bound, a), (step, wb, sl) in zip(outs, steps):
            agree(got[a], ref, bound + u_out * (np.abs(ref) + bound), "out")
            if decay is None:
                np.testing.assert_array_equal(w[sl], w0[sl])
            else:
                want = decay * w0[sl] + step
                agree(w[sl], want, wb + 2 * R.F32_U * (np.abs(want) + wb), "weight")
    return got, w


def seen_buckets(p):
    """Position and time buckets that the first sequence's pairs meet, by how often."""
    sl = slice(int(p.rows[0]), int(p.rows[0] + p.lens[0]))
    dp = np.clip(int(p.cand_pos[0]) - p.c.pos[sl].cpu().numpy().astype(np.int64), 0,
                 p.rab_p.shape[-1] - 1)
    bt = R.time_bucket(p.t[:p.n[0], None] - p.c.times[sl].cpu().numpy()[None], p.sub,
                       p.rab_t.shape[-1])
    order = lambda x: [b for _, b in sorted(zip(*np.unique(x, return_counts=True)[::-1]))]
    return order(dp), order(bt)


def problem(n, d, dtype, t_cand, seed):
    return Problem([300, 0, 40], [n, 5, 3], 2, d, d, dtype, seed=seed, nb=(40, 400),
                   t_cand=t_cand)


KINDS = [("bf16", "auto", n) for n in (8, 20, 64, 70, 130)] + [("bf16", "simt", 20),
                                                               ("f32", "auto", 20)]


@pytest.mark.parametrize("dtype,impl,n", KINDS)
@pytest.mark.parametrize("t_cand", [None, "apart"])
def test_a_nan_table_entry_reaches_its_pairs_and_no_other(dtype, impl, n, t_cand):
    for table in ("rab_p", "rab_t"):
        p = problem(n, 128, dtype, t_cand, 540 + n)
        pos, tim = seen_buckets(p)
        getattr(p, table)[pos[1] if table == "rab_p" else tim[0]] = np.nan
        got, w = check_values(p, impl=impl)
        assert np.isnan(got).any() and np.isnan(w).any()


@pytest.mark.parametrize("dtype,impl,n", KINDS)
@pytest.mark.parametrize("t_cand", [None, "apart"])
def test_a_nan_query_reaches_its_row_and_every_weight(dtype, impl, n, t_cand):
    for i in (0, 1, 2, 3, n - 1):
        p = problem(n, 64, dtype, t_cand, 550 + n)
        p.q[i, 1, 2] = float("nan")
        got, w = check_values(p, impl=impl)
        sl = slice(int(p.rows[0]), int(p.rows[0] + p.lens[0]))
        assert np.isnan(w[sl]).all() and np.isnan(got[i, 1]).all()


@pytest.mark.parametrize("dtype,impl,n", KINDS)
@pytest.mark.parametrize("t_cand", [None, "apart"])
def test_an_infinite_table_entry_gives_infinite_weights(dtype, impl, n, t_cand):
    """A tile's padding has the bias of its keys: it must not turn inf into NaN,
    which a trim would drop first instead of keeping."""
    for table in ("rab_p", "rab_t"):
        p = problem(n, 128, dtype, t_cand, 560 + n)
        pos, tim = seen_buckets(p)
        getattr(p, table)[pos[1] if table == "rab_p" else tim[0]] = np.inf
        got, w = check_values(p, impl=impl)
        assert np.isposinf(w).any()


# The weight-free form against the bounds of float32 arithmetic with P rounded to
# bf16 and nothing else: every way a tile finds its time bias, both tile widths.
FORMS = [dict(), dict(t_cand="apart", nb=(40, 400)), dict(t_cand="before", nb=(40, 400)),
         dict(t_cand="apart", sub=8, nb=(5000, 3000)), dict(t_cand="before", sub=8, nb=(50, 3000)),
         dict(t_cand="apart", t_step=10 ** 11, nb=(40, 400)), dict(t_cand="apart", sub=0),
         dict(per_head=True, t_cand="apart", nb=(1000, 1000), sub=4), dict(pad=5, shift=1),
         dict(alpha=-3.0)]


@pytest.mark.parametrize("decay", [None, 0.75])
@pytest.mark.parametrize("n", [7, 20, 64, 70, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", FORMS, ids=str)
def test_float32_arithmetic_with_and_without_weights(decay, n, d, kw):
    check_values(Problem([260, 33, 0, 129], [n, 9, 2, n], 2, d, d, "bf16", seed=570 + n, **kw),
                 decay)


@pytest.mark.parametrize("decay", [None, 0.75])
@pytest.mark.parametrize("n", [7, 20, 128])
@pytest.mark.parametrize("logit", [-3.0, -6.0, -12.0, -30.0, -88.0, -1000.0, 20.0, 200.0])
def test_logits_far_from_zero(decay, n, logit):
    """SiLU of a negative logit is small against the logit: a sigmoid with an absolute
    error would show."""
    p = Problem([260, 40], [n, 3], 2, 128, 128, "bf16", seed=580 + n, t_cand="apart",
                nb=(40, 400))
    p.rab_p += np.float32(logit)
    check_values(p, decay)


@pytest.mark.parametrize("decay", [None, 0.75])
@pytest.mark.parametrize("dtype,impl,n", KINDS)
@pytest.mark.parametrize("logit", [-6.5, -7.5, -8.9, -11.3, -14.1, -16.3, -19.7, -40.1, -79.0,
                                   1.7, 9.3])
def test_silu_is_good_to_a_part_of_itself(decay, dtype, impl, n, logit):
    """With alpha = 0 the bias is the logit, exactly, and P may be off by its
    rounding alone, however small it is: 2^-20 and the rounding of the exponential's
    argument, |x| (2^-24 + 2^-25), of itself, and for the tensor cores' product a
    twentieth more than half a step of bf16."""
    p = Problem([260, 33], [n, 9], 2, 64, 64, dtype, seed=600 + n, alpha=0.0)
    p.rab_p[:] = logit
    p.rab_t[:] = 0.0
    tc = dtype == "bf16" and impl == "auto"
    u = 2.0 ** -20 + abs(logit) * 2.0 ** -23
    w0 = p.c.weight.clone()
    got, w = run(p, decay, w0, impl=impl)
    got, w, w0 = f64(got), f64(w), f64(w0)
    u_out = R.BF16_U if dtype == "bf16" else R.F32_U
    for (_, _, a, (ref, bound, _, _)), (_, sl, _, (_, _, step, wb)) in zip(
            p.reference((u + (1.05 * R.BF16_U if tc else 0.0), 0.0, 0.0)),
            p.reference((u, 0.0, 0.0))):
        agree(got[a], ref, bound + u_out * (np.abs(ref) + bound), "out")
        if decay is not None:
            want = decay * w0[sl] + step
            agree(w[sl], want, wb + 2 * R.F32_U * (np.abs(want) + wb), "weight")


HIDING = ["far", "times", "own", "all"]


@pytest.mark.parametrize("dtype,impl,n", KINDS)
@pytest.mark.parametrize("t_cand", [None, "apart", "before"])
@pytest.mark.parametrize("hide", HIDING)
def test_a_hidden_bucket_hides_whatever_the_candidate_holds(dtype, impl, n, t_cand, hide):
    """A pair in a hidden bucket adds nothing: not the infinity or NaN of a query's
    dot product, nor 0 times the candidate's own infinite v.  Rows that a bad
    candidate does not see keep the weights, and rows of out the bits, that they
    have with an ordinary one."""
    for low in (-np.inf, float(np.finfo(np.float32).min)):
        p = problem(n, 64, dtype, t_cand, 620 + n)
        pos, tim = seen_buckets(p)
        if hide == "far":
            p.rab_p[39] = low               # (all positions from 39 on)
        elif hide == "times":
            p.rab_t[tim[::2]] = low
            p.rab_t[0] = 0.1
        elif hide == "own":
            p.rab_p[0] = low
        else:
            p.rab_p[:] = low
        w0 = p.c.weight.clone()
        for decay in (0.5, None):
            clean, w_clean = run(p, decay, w0, impl=impl)
            assert torch.isfinite(clean.float()).all()
            for i in sorted({0, 3, n - 1}):
                for bad in (float("inf"), float("nan")):
                    kept = p.q[i, 1].clone()
                    p.q[i, 1, 3] = bad
                    got, w = run(p, decay, w0, impl=impl)
                    p.q[i, 1] = kept
                    sl = slice(int(p.rows[0]), int(p.rows[0] + p.lens[0]))
                    dp = np.clip(int(p.cand_pos[0]) - p.c.pos[sl].cpu().numpy().astype(np.int64),
                                 0, 39)
                    bt = R.time_bucket(p.t[i] - p.c.times[sl].cpu().numpy(), p.sub, 400)
                    seen = (p.rab_p[dp] > -1e30) & (p.rab_t[bt] > -1e30)
                    own = p.rab_p[0] > -1e30 and p.rab_t[0] > -1e30
                    if seen.any() or own:
                        assert not torch.isfinite(got[i, 1].float()).any()
                        got[i, 1] = clean[i, 1]
                    assert torch.equal(bits(got), bits(clean)), (i, bad, decay)
                    if decay is not None:
                        hit = torch.from_numpy(seen).cuda()
                        assert not torch.isfinite(w[sl][hit]).any()
                        w[sl] = torch.where(hit, w_clean[sl], w[sl])
                    assert torch.equal(bits(w), bits(w_clean)), (i, bad)
            if not (p.rab_p[0] > -1e30):
                for bad in (float("inf"), float("nan")):
                    kept = p.v[1, 1].clone()
                    p.v[1, 1, 3] = bad
                    got, _ = run(p, decay, w0, impl=impl)
                    p.v[1, 1] = kept
                    assert torch.equal(bits(got), bits(clean)), bad


@pytest.mark.parametrize("n", [5, 20, 100])
@pytest.mark.parametrize("decay", [0.5, None])
def test_own_values_with_the_keys_split_over_ctas(n, decay):
    """Only the first key range adds the own pairs: the summing pass must see them once."""
    p = Problem([6000, 2500], [n, 3], 1, 128, 128, "bf16", seed=640 + n)
    check_values(p, decay)
    w0 = p.c.weight.clone()
    clean, w_clean = run(p, decay, w0)
    p.v[n // 2, 0, 9] = float("inf")
    got, w = run(p, decay, w0)
    assert not torch.isfinite(got[n // 2, 0, 9])
    got[n // 2, 0, 9] = clean[n // 2, 0, 9]
    assert torch.equal(bits(got), bits(clean)) and torch.equal(bits(w), bits(w_clean))


@pytest.mark.parametrize("n", [8, 40, 130])
def test_a_nan_row_through_the_layer(n):
    """One candidate's NaN input reaches its own row of the projection and of y."""
    H, d, D = 2, 128, 64
    rng = np.random.default_rng(650 + n)
    p = Problem([260, 0], [n, 4], H, d, d, "bf16", seed=651)
    P = layer_params(rng, H, d, D)
    x = torch.from_numpy(rng.standard_normal((n + 4, D)).astype(np.float32)).cuda().bfloat16()

    def layer():
        proj = torch.empty((n + 4, 4 * H * d), dtype=torch.bfloat16, device="cuda")
        y = ops.layer_fwd_candidates_qcache(
            x, *P, p.c, p.rows, p.lens, p.off, p.cand_pos, p.ts, num_heads=H, d_qk=d, d_v=d,
            max_seq_len=p.msl, time_bucket_sub_bits=2, silu_scale=p.scale, proj_out=proj)
        return y, proj
    y0, proj0 = layer()
    for i in (0, n - 1, n + 1):
        kept = x[i].clone()
        x[i] = float("nan")
        y, proj = layer()
        x[i] = kept
        assert torch.isnan(y[i]).all() and torch.isnan(proj[i]).all()
        y[i], proj[i] = y0[i], proj0[i]
        assert torch.equal(bits(y), bits(y0)) and torch.equal(bits(proj), bits(proj0))


def test_a_captured_step_appends_scores_and_trims():
    """Events stored, candidates scored with weights and the histories trimmed in one
    graph: each replay does what the calls one behind the other do."""
    H, d, D = 2, 64, 64
    rng = np.random.default_rng(660)
    p = Problem([300, 90], [33, 2], H, d, d, "bf16", seed=661)
    P = layer_params(rng, H, d, D)
    x = torch.from_numpy(rng.standard_normal((35, D)).astype(np.float32)).cuda().bfloat16()
    FIELDS = ("k_codes", "k_scales", "v_codes", "v_scales", "times", "pos", "weight")
    start = {f: getattr(p.c, f).clone() for f in FIELDS}
    y = torch.empty((35, D), dtype=torch.bfloat16, device="cuda")
    proj = torch.empty((35, 4 * H * d), dtype=torch.bfloat16, device="cuda")
    F = H * d
    pick = torch.tensor([0, 33], device="cuda")

    def step():
        ops.layer_fwd_candidates_qcache(
            x, *P, p.c, p.rows, p.lens, p.off, p.cand_pos, p.ts, num_heads=H, d_qk=d, d_v=d,
            max_seq_len=p.msl + 2, time_bucket_sub_bits=2, silu_scale=p.scale, weight_decay=0.5,
            proj_out=proj, out=y)
        ev = proj[pick]
        ops.qcache_append(p.c, ev[:, 3 * F:], ev[:, F:2 * F], p.ts[pick], [0, 1, 2],
                          p.rows + p.lens, p.cand_pos)
        ops.qcache_evict(p.c, p.rows, p.lens + 1, [200, 50], p.cand_pos - 4)

    def reset():
        for f in FIELDS:
            getattr(p.c, f).copy_(start[f])
    step()
    want = [y.clone(), proj.clone()] + [getattr(p.c, f).clone() for f in FIELDS]
    reset()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g):
            step()
    for _ in range(2):
        torch.cuda.synchronize()
        reset()
        y.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = [y, proj] + [getattr(p.c, f) for f in FIELDS]
        for a, b in zip(got, want):
            same = a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)
            assert torch.equal(*same)


@pytest.mark.parametrize("decay", [None, 0.5])
@pytest.mark.parametrize("H,d,L,n", [(2, 64, 20, 5), (2, 64, 20, 20), (2, 64, 20, 100),
                                     (1, 128, 20, 40), (4, 32, 20, 20), (2, 64, 600, 5),
                                     (2, 64, 900, 70), (1, 32, 3000, 3)])
def test_layer_norm_sees_the_attention_in_float32(decay, H, d, L, n):
    """Attention outputs whose features differ by little against their size: the
    LayerNorm takes the size away and leaves a rounding of it magnified.

    All keys share one v row of 12..15 eighths, alpha is 0 and the own pair hidden, so
    the attention is a multiple of that row (whatever P's rounding) and the LayerNorm
    is known.  W2 is the identity: y is g, rounded once.  The bound: that rounding, and
    float32 sums over keys (2 u a term) and features (u a term) against the deviation."""
    F = H * d
    rng = np.random.default_rng(670 + n)
    p = Problem([L, 7], [n, 3], H, d, d, "bf16", seed=671)
    P = list(layer_params(rng, H, d, F))
    P[4] = torch.eye(F, dtype=torch.bfloat16, device="cuda")
    P[5] = torch.zeros(F, device="cuda")
    P[6] = P[6] + 1.0
    P[6][0] = float("-inf")
    v_row = (12 + rng.integers(0, 4, (1, H, d))) / 8.0
    for b in range(2):
        m = int(p.lens[b])
        vt = torch.from_numpy(np.repeat(v_row, m, 0).astype(np.float32)).cuda().bfloat16()
        t, pos = p.c.times.clone(), p.c.pos.clone()
        kt, _ = ops.qcache_read(p.c, [p.rows[b]], [m])
        ops.qcache_append(p.c, kt, vt, torch.zeros(m, dtype=torch.int64, device="cuda"), [0, m],
                          [p.rows[b]], [0])
        p.c.times.copy_(t)
        p.c.pos.copy_(pos)
    x = torch.from_numpy(rng.standard_normal((n + 3, F)).astype(np.float32)).cuda().bfloat16()
    proj = torch.empty((n + 3, 4 * F), dtype=torch.bfloat16, device="cuda")
    y = f64(ops.layer_fwd_candidates_qcache(
        x, *P, p.c, p.rows, p.lens, p.off, p.cand_pos, p.ts, num_heads=H, d_qk=d, d_v=d,
        max_seq_len=p.msl, time_bucket_sub_bits=2, alpha=0.0, silu_scale=1.0, residual=False,
        proj_out=proj, weight_decay=decay))
    u, _, q, k = (f64(proj)[:, i * F:(i + 1) * F].reshape(-1, H, d) for i in range(4))
    rp, rt = f64(P[6]), f64(P[7])
    ga, be = f64(P[2]), f64(P[3])
    for b in range(2):
        sl, a = slice(int(p.rows[b]), int(p.rows[b] + p.lens[b])), \
            slice(int(p.off[b]), int(p.off[b + 1]))
        kh, vh = stored(p.c, p.rows[b], p.lens[b])
        np.testing.assert_array_equal(vh, np.repeat(v_row, int(p.lens[b]), 0))
        with np.errstate(invalid="ignore"):      # (the bound of the hidden own pair)
            out, _, _, _ = R.attend(q[a], k[a], np.zeros_like(q[a]), kh, vh,
                                    p.c.pos[sl].cpu().numpy(), p.c.times[sl].cpu().numpy(),
                                    int(p.cand_pos[b]), p.t[a], rp, rt, 2, 0.0, 1.0, 0.0)
        A = out.reshape(-1, F)
        mu, sd = A.mean(1, keepdims=True), np.sqrt(A.var(1, keepdims=True) + 1e-5)
        ln = (A - mu) / sd
        assert np.all(np.abs(mu) > 3 * sd)
        err = 2 ** -23 * (int(p.lens[b]) + 8 + F) * np.abs(A).max(1, keepdims=True)
        dln = 2 * err / sd * (1 + np.abs(ln)) + 2.0 ** -20 * (1 + np.abs(ln))
        g = (ln * ga + be) * u[a].reshape(-1, F)
        tol = np.abs(u[a].reshape(-1, F)) * np.abs(ga) * dln
        assert np.all(np.abs(y[a] - g) <= tol + R.BF16_U * (np.abs(g) + tol)), \
            float((np.abs(y[a] - g) / (np.abs(g) + 1e-3)).max())


@pytest.mark.parametrize("decay", [None, 0.0])
@pytest.mark.parametrize("dtype,impl,n", KINDS)
@pytest.mark.parametrize("t_cand", [None, "apart"])
def test_rows_of_which_nothing_is_left_are_zero(decay, dtype, impl, n, t_cand):
    for table in ("rab_p", "rab_t"):
        p = problem(n, 128, dtype, t_cand, 690 + n)
        getattr(p, table)[:] = -np.inf
        got, w = run(p, decay, p.c.weight.clone(), impl=impl)
        assert torch.all(got == 0)
        if decay is not None:
            for b in range(3):
                assert torch.all(w[p.rows[b]:p.rows[b] + p.lens[b]] == 0)


@pytest.mark.parametrize("H,dk,dv,n", [(2, 64, 32, 5), (2, 64, 32, 40), (1, 32, 128, 3),
                                       (4, 128, 64, 20), (2, 96, 64, 9)])
def test_layer_of_unequal_key_and_value_sizes(H, dk, dv, n):
    """The columns [U|V|Q|K] of the projection, by the attention on views of it."""
    rng = np.random.default_rng(680 + n)
    p = Problem([300, 0, 41], [n, 2, 1], H, dk, dv, "bf16", seed=681)
    T, D, F = n + 3, 64, H * dv
    n1 = 2 * (F + H * dk)
    w = lambda *s: torch.from_numpy((rng.standard_normal(s) / 8).astype(np.float32)).cuda()
    w1, w2 = w(n1, D).bfloat16(), w(D, F).bfloat16()
    b1, ga, be, b2, rp, rt = w(n1), 1 + w(F), w(F), w(D), w(40), w(24)
    x = (8 * w(T, D)).bfloat16()
    proj = torch.empty((T, n1), dtype=torch.bfloat16, device="cuda")
    kw = dict(max_seq_len=p.msl, time_bucket_sub_bits=2, silu_scale=p.scale)
    y = ops.layer_fwd_candidates_qcache(
        x, w1, b1, ga, be, w2, b2, rp, rt, p.c, p.rows, p.lens, p.off, p.cand_pos, p.ts,
        num_heads=H, d_qk=dk, d_v=dv, proj_out=proj, **kw)
    v, q, k = (proj[:, a:b] for a, b in ((F, 2 * F), (2 * F, 2 * F + H * dk), (2 * F + H * dk, n1)))
    u_in = f64(x) @ f64(w1).T + f64(b1)
    z = u_in / (1 + np.exp(-u_in))
    # (half a step of bf16, and as much again with 1e-4 for float32 sums and the tanh)
    assert np.all(np.abs(f64(proj) - z) <= 2.0 ** -7 * np.abs(z) + 1e-4)
    q, k, v, u = (f64(t).reshape(T, H, -1) for t in (q, k, v, proj[:, :F]))
    A = np.zeros((T, F))
    for b in range(3):
        a, sl = slice(int(p.off[b]), int(p.off[b + 1])), \
            slice(int(p.rows[b]), int(p.rows[b] + p.lens[b]))
        kh, vh = stored(p.c, p.rows[b], p.lens[b])
        A[a] = R.attend(q[a], k[a], v[a], kh, vh, p.c.pos[sl].cpu().numpy(),
                        p.c.times[sl].cpu().numpy(), int(p.cand_pos[b]), p.t[a], f64(rp), f64(rt),
                        2, 1 / np.sqrt(dk), p.scale, 0.0)[0].reshape(-1, F)
    mu = A.mean(1, keepdims=True)
    g = (A - mu) / np.sqrt(((A - mu) ** 2).mean(1, keepdims=True) + 1e-5) * f64(ga) + f64(be)
    want = f64(x) + (g * u.reshape(T, F)) @ f64(w2).T + f64(b2)
    assert_close(f64(y), want, "bf16", "layer")
