"""The 4-bit history cache on the CPU: the format's reference against brute
force, and the entry points' refusals, which come before any CUDA call (run in
a process that sees no device, like the other refusal tests)."""
import ctypes
import multiprocessing as mp
import os

import numpy as np
import pytest

from hstu_pointwise_attention_b200 import ops

import qcache_ref as R

OK, INVALID, UNSUPPORTED, WORKSPACE, CUDA = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def hidden():
    old = os.environ.get("CUDA_VISIBLE_DEVICES")
    os.environ["CUDA_VISIBLE_DEVICES"] = ""
    try:
        pool = mp.get_context("spawn").Pool(1)
    finally:
        if old is None:
            del os.environ["CUDA_VISIBLE_DEVICES"]
        else:
            os.environ["CUDA_VISIBLE_DEVICES"] = old
    yield pool
    pool.close()
    pool.join()


# ---- the format ----
def test_format_is_the_best_code_on_its_grid():
    """Scale, zero point and codes from their definition, by search."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((6, 2, 64)) * np.exp2(rng.integers(-20, 20, (6, 2, 1)))
    x[0] = np.abs(x[0])
    x[1] = -np.abs(x[1])
    x[2, 0, :32] = 0.0
    q, s, z = R.quantise(x)
    for t in range(6):
        for h in range(2):
            for g in range(2):
                v = x[t, h, 32 * g:32 * g + 32]
                span = max(v.max(), 0) - min(v.min(), 0)
                if span == 0:
                    assert s[t, h, g] == 0 and z[t, h, g] == 0
                    continue
                e = int(np.floor(np.log2(span / 15)))
                grid = [m / 8 * 2.0 ** k for k in (e - 1, e, e + 1) for m in range(8, 16)]
                assert s[t, h, g] == min(c for c in grid if 15 * c >= span)
                dq = R.values(q, s, z)[t, h, 32 * g:32 * g + 32]
                assert np.all(np.abs(dq - v) <= s[t, h, g] / 2)
                assert np.all(dq[v == 0] == 0)


def test_pack_and_unpack_agree_and_values_are_bf16():
    rng = np.random.default_rng(6)
    q, s, z = R.quantise(rng.standard_normal((5, 3, 96)))
    codes, params = R.pack(q, s, z)
    got = R.unpack(codes, params)
    np.testing.assert_array_equal(got, R.values(q, s, z))
    bits = got.astype(np.float32).view(np.uint32)
    assert np.all(bits & 0xFFFF == 0)


def test_reference_bound_covers_a_float32_evaluation():
    """The stated error bound holds for a plain float32 evaluation."""
    rng = np.random.default_rng(7)
    n, H, d, L = 3, 2, 32, 50
    a = [rng.standard_normal((m, H, d)).astype(np.float32) for m in (n, n, n, L, L)]
    pos, t = np.arange(L), np.arange(L) * 100
    rp, rt = (rng.standard_normal(16).astype(np.float32) for _ in range(2))
    args = (pos, t, L, np.full(n, 100 * L), rp, rt, 0, 0.2, 0.1)
    out, bound, w, wb = R.attend(*[x.astype(np.float64) for x in a], *args, u_p=8 * R.F32_U)
    dp = np.clip(L - pos, 0, 15)
    bt = R.time_bucket(100 * L - t, 0, 16)
    for h in range(H):
        x = np.float32(0.2) * (a[0][:, h] @ a[3][:, h].T) + rp[dp] + rt[bt]
        p = x / (1 + np.exp(-x, dtype=np.float32))
        xs = np.float32(0.2) * (a[0][:, h] * a[1][:, h]).sum(1) + rp[0] + rt[0]
        got = np.float32(0.1) * (p @ a[4][:, h] + (xs / (1 + np.exp(-xs)))[:, None] * a[2][:, h])
        assert np.all(np.abs(got - out[:, h]) <= bound[:, h] + R.F32_U * np.abs(out[:, h]))


# ---- refusals ----
def _cache(rows=64, H=2, dk=64, dv=64, **kw):
    c = ops._QCacheStruct(rows, H, dk, dv, 0, *([4096] * 7))
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _i64(*a):
    return np.array(a, np.int64)


def _i32(*a):
    return np.array(a, np.int32)


def _hidden():
    return os.environ.get("CUDA_VISIBLE_DEVICES") == ""


def _append(cache=None, dtype=1, B=2, off=(0, 3, 5), rows=(0, 10), pos=(0, 0), k=4096, krs=128,
            v=4096, vrs=128, ts=4096):
    assert _hidden()
    off, rows, pos = _i64(*off), _i64(*rows), _i32(*pos)
    return ops.LIB.hstu_qcache_append(ctypes.byref(cache or _cache()), dtype, B, off.ctypes.data,
                                      rows.ctypes.data, pos.ctypes.data, k, krs, v, vrs, ts, None)


def _append_cases():
    I = INVALID
    bad = [
        (I, dict(dtype=7)), (I, dict(B=-1)), (I, dict(off=(1, 3, 5))), (I, dict(off=(0, 5, 3))),
        (I, dict(rows=(-1, 10))), (I, dict(rows=(0, 63))), (I, dict(rows=(0, 2))),
        (I, dict(rows=(10, 9))), (I, dict(krs=127)), (I, dict(vrs=0)), (I, dict(k=None)),
        (I, dict(v=None)), (I, dict(ts=None)), (I, dict(k=4097)), (I, dict(ts=4100)),
        (I, dict(pos=(2 ** 31 - 2, 0))), (UNSUPPORTED, dict(cache=_cache(rows=2 ** 33),
                                                            off=(0, 2 ** 31, 2 ** 31),
                                                            rows=(0, 2 ** 32))),
        (I, dict(cache=_cache(H=0))), (I, dict(cache=_cache(dk=48))),
        (I, dict(cache=_cache(dv=288))), (I, dict(cache=_cache(rows=-1))),
        (I, dict(cache=_cache(k_codes=4104))), (I, dict(cache=_cache(v_codes=None))),
        (I, dict(cache=_cache(k_scales=4097))), (I, dict(cache=_cache(times=None))),
        (I, dict(cache=_cache(pos=None))), (I, dict(cache=_cache(weight=4098)))]
    fine = [(OK, dict(off=(0, 0, 0))), (OK, dict(B=0)), (CUDA, dict()),
            (CUDA, dict(cache=_cache(weight=None))), (CUDA, dict(rows=(10, 0))),
            (CUDA, dict(rows=(10, 8)))]
    return [(want, _append(**kw), str(sorted(kw))) for want, kw in bad + fine]


def _read(cache=None, dtype=1, B=2, rows=(0, 0), lens=(3, 64), k=4096, krs=128, v=4096, vrs=128):
    assert _hidden()
    rows, lens = _i64(*rows), _i64(*lens)
    return ops.LIB.hstu_qcache_read(ctypes.byref(cache or _cache()), dtype, B, rows.ctypes.data,
                                    lens.ctypes.data, k, krs, v, vrs, None)


def _read_cases():
    I = INVALID
    bad = [(I, dict(dtype=2)), (I, dict(B=-1)), (I, dict(rows=(0, 1))), (I, dict(lens=(-1, 2))),
           (I, dict(rows=(-1, 0))), (I, dict(krs=64)), (I, dict(vrs=64)), (I, dict(k=None)),
           (I, dict(v=4097)), (I, dict(cache=_cache(dk=0)))]
    fine = [(OK, dict(lens=(0, 0))), (CUDA, dict())]
    return [(want, _read(**kw), str(sorted(kw))) for want, kw in bad + fine]


def _attn_params(B=2, H=2, dk=64, dv=64, msl=64, **kw):
    p = ops.AttnParams()
    p.batch, p.num_heads, p.d_qk, p.d_v, p.max_seq_len = B, H, dk, dv, msl
    p.num_pos_buckets = p.num_time_buckets = 32
    p.time_bucket_sub_bits = 2
    p.dtype = ops.BF16
    for f in ("q", "k", "v", "o"):
        setattr(p, f + "_row_stride", H * max(dk, dv))
    p.alpha, p.silu_scale = 0.125, 1.0 / 64
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def _attn(p=None, cache=None, rows=(0, 32), lens=(20, 30), coff=(0, 3, 5), pos=(20, 30), ts=4096,
          q=4096, k=4096, v=4096, rp=4096, rt=4096, upd=1, decay=0.5, out=4096, ws=4096,
          nbytes=None):
    assert _hidden()
    p = p or _attn_params()
    rows, lens, coff, pos = _i64(*rows), _i64(*lens), _i64(*coff), _i32(*pos)
    n = ctypes.c_size_t(0)
    rc = ops.LIB.hstu_attn_candidates_qcache_workspace_size(
        ctypes.byref(p), lens.ctypes.data, coff.ctypes.data, upd, ctypes.byref(n))
    if nbytes is None:
        nbytes = n.value if rc == OK else 1 << 30
    return ops.LIB.hstu_attn_fwd_candidates_qcache(
        ctypes.byref(p), ctypes.byref(cache or _cache()), rows.ctypes.data, lens.ctypes.data,
        coff.ctypes.data, pos.ctypes.data, ts, q, k, v, rp, rt, upd, decay, out, ws, nbytes, None)


def _attn_cases():
    I = INVALID
    P = _attn_params
    bad = [
        (I, dict(p=P(H=3))), (I, dict(p=P(dk=32))), (I, dict(p=P(dk=48), cache=_cache(dk=48))),
        (I, dict(p=P(B=-1))), (I, dict(p=P(msl=31))), (I, dict(p=P(num_pos_buckets=0))),
        (I, dict(p=P(time_bucket_sub_bits=9))), (I, dict(p=P(dtype=3))),
        (I, dict(p=P(q_row_stride=127))), (I, dict(p=P(o_row_stride=1))),
        (I, dict(p=P(alpha=float("nan")))), (I, dict(rows=(0, 40))), (I, dict(rows=(-1, 32))),
        (I, dict(lens=(-1, 30))), (I, dict(rows=(0, 19))), (I, dict(coff=(0, 4, 3))),
        (I, dict(coff=(1, 4, 5))), (I, dict(decay=float("inf"))),
        (I, dict(cache=_cache(weight=None))), (I, dict(ts=None)), (I, dict(q=None)),
        (I, dict(k=None)), (I, dict(v=None)), (I, dict(rp=None)), (I, dict(rt=None)),
        (I, dict(out=None)), (I, dict(q=4097)), (I, dict(out=4097)), (I, dict(ts=4100)),
        (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws=4096 + 128)),
        (WORKSPACE, dict(nbytes=16))]
    fine = [(CUDA, dict()), (CUDA, dict(rows=(0, 19), upd=0)),
            (CUDA, dict(cache=_cache(weight=None), upd=0)),
            (CUDA, dict(p=P(msl=32))), (CUDA, dict(lens=(0, 0)))]
    return [(want, _attn(**kw), str(sorted(kw))) for want, kw in bad + fine]


def _evict(src=None, dst=None, B=2, rows=(0, 32), lens=(20, 30), budgets=(10, 40), keep=(5, 5),
           to=(0, 32), ws=1 << 20, nbytes=1 << 20):
    assert _hidden()
    src = src or _cache()
    rows, lens, budgets, keep, to = (_i64(*rows), _i64(*lens), _i64(*budgets), _i32(*keep),
                                     _i64(*to))
    return ops.LIB.hstu_qcache_evict(ctypes.byref(src), ctypes.byref(dst or src), B,
                                     rows.ctypes.data, lens.ctypes.data, budgets.ctypes.data,
                                     keep.ctypes.data, to.ctypes.data, ws, nbytes, None)


def _other(**kw):
    c = _cache(**kw)
    for i, f in enumerate(("k_codes", "k_scales", "v_codes", "v_scales", "times", "pos",
                           "weight")):
        setattr(c, f, (1 << 24) + (i << 20))
    return c


def _evict_cases():
    I = INVALID
    partly = _other()
    partly.v_scales = 4096
    inside = _other()
    inside.k_codes = 4096 + 2 * 64 * 32 - 16
    bad = [(I, dict(lens=(-1, 30))), (I, dict(budgets=(-1, 2))), (I, dict(rows=(0, 40))),
           (I, dict(rows=(0, 10), to=(0, 10))), (I, dict(to=(1, 32))),
           (I, dict(src=_cache(weight=None))), (I, dict(dst=_other(H=4))),
           (I, dict(dst=_other(dk=32))),
           (I, dict(dst=_other(), to=(0, 9))), (I, dict(dst=_other(), to=(0, 40))),
           (I, dict(dst=partly)), (I, dict(dst=inside)),
           (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(nbytes=64)),
           (WORKSPACE, dict(ws=(1 << 20) + 16))]
    fine = [(OK, dict(lens=(0, 0))), (OK, dict(budgets=(20, 30))), (OK, dict(budgets=(0, 0))),
            (CUDA, dict()), (CUDA, dict(dst=_other(), to=(40, 0)))]
    return [(want, _evict(**kw), str(sorted(kw))) for want, kw in bad + fine]


def _layer(D=64, upd=0, x=4096, y=8192, proj=None, dtype=1, H=2, ln_eps=1e-5, ws=4096,
           nbytes=1 << 30):
    assert _hidden()
    lp = ops.LayerParams()
    lp.attn = _attn_params(H=H, dtype=dtype)
    lp.d_model, lp.residual, lp.ln_eps = D, 1, ln_eps
    rows, lens, coff, pos = _i64(0, 32), _i64(20, 30), _i64(0, 3, 5), _i32(20, 30)
    return ops.LIB.hstu_layer_fwd_candidates_qcache(
        ctypes.byref(lp), ctypes.byref(_cache(H=H)), rows.ctypes.data, lens.ctypes.data,
        coff.ctypes.data, pos.ctypes.data, *([4096] * 1), x, *([4096] * 8), upd, 0.5, y, proj, ws,
        nbytes, None)


def _layer_cases():
    I = INVALID
    bad = [(I, dict(D=60)), (I, dict(D=0)), (I, dict(x=None)), (I, dict(y=None)),
           (I, dict(y=4096)), (I, dict(proj=4104)), (I, dict(ln_eps=0.0)),
           (UNSUPPORTED, dict(dtype=0)), (UNSUPPORTED, dict(H=3)), (WORKSPACE, dict(nbytes=1024)),
           (WORKSPACE, dict(ws=None))]
    return [(want, _layer(**kw), str(sorted(kw))) for want, kw in bad + [(CUDA, dict())]]


@pytest.mark.parametrize("cases", [_append_cases, _read_cases, _attn_cases, _evict_cases,
                                   _layer_cases])
def test_refusals(hidden, cases):
    wrong = [c for c in hidden.apply(cases) if c[0] != c[1]]
    assert not wrong, wrong


def _sizes():
    assert _hidden()
    out = []
    p = _attn_params(msl=1 << 20)
    for lens, coff, upd in [((0, 0), (0, 0, 0), 1), ((1, 1), (0, 1, 2), 0),
                            ((100000, 5), (0, 1, 2), 1), ((100000, 5), (0, 300, 301), 1)]:
        lens, coff, n = _i64(*lens), _i64(*coff), ctypes.c_size_t(0)
        rc = ops.LIB.hstu_attn_candidates_qcache_workspace_size(
            ctypes.byref(p), lens.ctypes.data, coff.ctypes.data, upd, ctypes.byref(n))
        out.append((rc, n.value))
    return out


def test_workspace_sizes(hidden):
    (a, none), (b, one), (c, long), (d, many) = hidden.apply(_sizes)
    assert a == b == c == d == OK
    assert 16 <= none <= one < long < many
    # one weight partial per cached row and head at least, 4 bytes each
    assert long >= 100000 * 2 * 4


def test_binding_refuses_before_the_library():
    import torch
    if torch.cuda.is_available():
        pytest.skip("checked with CPU tensors only")
    z = lambda *s, dt=torch.uint8: torch.zeros(s, dtype=dt)
    good = dict(k_codes=z(2, 8, 32), k_scales=z(2, 8, 2, dt=torch.int16), v_codes=z(2, 8, 32),
                v_scales=z(2, 8, 2, dt=torch.int16), times=z(8, dt=torch.int64),
                pos=z(8, dt=torch.int32), weight=z(8, dt=torch.float32))
    c = ops.QuantCache(**good)
    assert (c.rows, c.num_heads, c.d_qk, c.d_v) == (8, 2, 64, 64)
    for name, bad in [("k_codes", z(2, 8, 32, dt=torch.int8)), ("k_scales", z(2, 8, 4, dt=torch.int16)),
                      ("v_codes", z(2, 9, 32)), ("times", z(8, dt=torch.int32)),
                      ("pos", z(7, dt=torch.int32)), ("weight", z(16, dt=torch.float32)[::2])]:
        with pytest.raises(ValueError):
            ops.QuantCache(**{**good, name: bad})
    k = torch.zeros(3, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):      # a CPU tensor never reaches a kernel
        ops.qcache_append(c, k, k, torch.zeros(3, dtype=torch.int64), [0, 3], [0], [0])
    with pytest.raises(ValueError):
        ops.qcache_append(c, k, k, torch.zeros(2, dtype=torch.int64), [0, 3], [0], [0])
    with pytest.raises(ValueError):
        ops.qcache_evict(c, [0], [4], [2], [0], dst=c)
