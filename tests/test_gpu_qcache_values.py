"""The 4-bit history cache's attention where its values are not ordinary:
infinities and NaN in a candidate or in a bias table, each of them kept to the
rows and sums that the definition gives it to."""
import numpy as np
import pytest
import torch

import qcache_ref as R
from test_gpu_qcache import Problem, f64

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
