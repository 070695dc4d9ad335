"""The 4-bit history cache's attention where its values are not ordinary:
infinities and NaN in a candidate or in a bias table, each of them kept to the
rows and sums that the definition gives it to."""
import numpy as np
import pytest
import torch

from test_gpu_qcache import Problem

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
