"""The 4-bit history cache on the CPU: calls at the edge of what its kernels index,
and calls that would race or read out of place, are refused before any launch (in a
process that sees no device, where an accepted call ends with the CUDA error)."""
import ctypes

import numpy as np
import pytest

from hstu_pointwise_attention_b200 import ops

from test_qcache_host import (CUDA, INVALID, OK, UNSUPPORTED, _attn, _attn_params, _cache, _evict,
                              _hidden, _i64, _other, hidden)  # noqa: F401

LONGEST = 2 ** 31 - 1024     # rows of a sequence: loops step int32 indices by up to 1,024


def wrong(cases):
    return [c for c in cases if c[0] != c[1]]


def _lengths():
    assert _hidden()
    out = []
    big = _cache(rows=2 ** 33, H=1, dk=32, dv=32)
    far = _cache(rows=2 ** 33, H=1, dk=32, dv=32)
    for i, (f, _) in enumerate(ops._QCacheStruct._fields_[5:]):
        setattr(far, f, (i + 2) << 44)
    for n in (LONGEST, LONGEST + 1, 2 ** 31 - 1):
        want = CUDA if n <= LONGEST else UNSUPPORTED
        kw = dict(src=big, rows=(0, 2 ** 32), to=(0, 2 ** 32), nbytes=1 << 40)
        out += [(want, _evict(lens=(n, 30), budgets=(1000, 10), **kw), f"in place {n}"),
                (want, _evict(lens=(30, n), budgets=(7, 1), dst=far, **kw), f"copied {n}")]
        size = ctypes.c_size_t(0)
        lens, budgets = _i64(n), _i64(5)
        out.append((OK if n <= LONGEST else UNSUPPORTED,
                    ops.LIB.hstu_qcache_evict_workspace_size(
                        1, lens.ctypes.data, budgets.ctypes.data, ctypes.byref(size)), f"size {n}"))
        for dtype in (0, 1):
            p = _attn_params(H=1, dk=32, dv=32, msl=2 ** 31 - 1, dtype=dtype)
            for upd in (0, 1):
                out.append((want, _attn(p=p, cache=big, rows=(0, 2 ** 32),
                                        lens=(n, 5), coff=(0, 0, 2), upd=upd, nbytes=1 << 50),
                            f"attention {n} {dtype} {upd}"))
    return out


def test_longest_sequences(hidden):  # noqa: F811
    assert not wrong(hidden.apply(_lengths))


def _candidate_totals():
    """Candidates times heads, which a launch counts in 32 bits, at sizes where the
    product leaves 64."""
    assert _hidden()
    B = 1 << 21
    n = 2 ** 31 - 1024
    p = _attn_params(B=B, H=4096, dk=32, dv=32, msl=2 ** 31 - 1)
    lens = np.zeros(B, np.int64)
    coff = np.arange(B + 1, dtype=np.int64) * n
    size = ctypes.c_size_t(0)
    return [(UNSUPPORTED, ops.LIB.hstu_attn_candidates_qcache_workspace_size(
        ctypes.byref(p), lens.ctypes.data, coff.ctypes.data, 0, ctypes.byref(size)), "total")]


def test_candidate_totals(hidden):  # noqa: F811
    assert not wrong(hidden.apply(_candidate_totals))


FIELDS = ("k_codes", "k_scales", "v_codes", "v_scales", "times", "pos", "weight")


def _apart(rows=64, H=2, d=64):
    """Two caches whose buffers lie apart, and every buffer's bytes."""
    size = dict(zip(FIELDS, (rows * H * d // 2, rows * H * d // 16) * 2 +
                    (rows * 8, rows * 4, rows * 4)))
    src, dst = _cache(rows=rows), _cache(rows=rows)
    for i, f in enumerate(FIELDS):
        setattr(src, f, (1 << 24) + (i << 20))
        setattr(dst, f, (2 << 24) + (i << 20))
    return src, dst, size


def _shared_memory():
    """A destination buffer that lies in any buffer of the source, at its first and
    its last bytes, is refused; right behind or ahead of it is fine."""
    out = []
    src, dst, size = _apart()
    out.append((CUDA, _evict(src=src, dst=dst), "apart"))
    for a in FIELDS:
        for b in FIELDS:
            base = getattr(src, a)
            for at, want in ((base, INVALID), (base + size[a] - 16, INVALID),
                             (base - size[b] + 16, INVALID), (base + size[a], CUDA),
                             (base - size[b], CUDA)):
                src, dst, _ = _apart()
                setattr(dst, b, at)
                out.append((want, _evict(src=src, dst=dst), (a, b, at - base)))
    src, dst, _ = _apart()
    dst.rows = 0                       # an empty cache shares nothing
    dst.k_codes = src.k_codes + 32
    out.append((OK, _evict(src=src, dst=dst, budgets=(0, 0), to=(0, 0)), "empty"))
    return out


def test_evict_refuses_any_shared_memory(hidden):  # noqa: F811
    assert not wrong(hidden.apply(_shared_memory))


LAYER_ARGS = ("ts", "x", "w1", "b1", "gamma", "beta", "w2", "b2", "rab_p", "rab_t")


def _layer_call(**kw):
    """A layer call on 5 candidates of d_model 64; every buffer can be placed."""
    assert _hidden()
    at = {n: (i + 1) << 24 for i, n in enumerate(LAYER_ARGS + ("y", "ws"))}
    at["proj"] = None
    at.update(kw)
    lp = ops.LayerParams()
    lp.attn = _attn_params()
    lp.d_model, lp.residual, lp.ln_eps = 64, 1, 1e-5
    rows, lens, coff, pos = _i64(0, 32), _i64(20, 30), _i64(0, 3, 5), np.array([20, 30], np.int32)
    return ops.LIB.hstu_layer_fwd_candidates_qcache(
        ctypes.byref(lp), ctypes.byref(_cache()), rows.ctypes.data, lens.ctypes.data,
        coff.ctypes.data, pos.ctypes.data, *(at[n] for n in LAYER_ARGS), 1, 0.5, at["y"],
        at["proj"], at["ws"], 1 << 24, None)


def _layer_alignment():
    out = [(CUDA, _layer_call(), "aligned")]
    for n in LAYER_ARGS + ("y",):
        size = 8 if n == "ts" else 2 if n in ("x", "w1", "w2", "y") else 4
        base = (20 << 24)
        out += [(INVALID, _layer_call(**{n: base + size // 2}), n),
                (CUDA, _layer_call(**{n: base + size}), n)]
    return out


def test_layer_refuses_buffers_off_their_elements(hidden):  # noqa: F811
    assert not wrong(hidden.apply(_layer_alignment))


def _layer_overlap():
    x, out = 20 << 24, []
    rows, proj = 5 * 64 * 2, 5 * 4 * 128 * 2            # bytes of x (or y) and of proj_out
    for at, want in ((x, INVALID), (x + rows - 16, INVALID), (x - rows + 16, INVALID),
                     (x + rows, CUDA), (x - rows, CUDA)):
        out.append((want, _layer_call(x=x, y=at), ("y on x", at - x)))
    for n in ("x", "y"):
        for at, want in ((x, INVALID), (x + rows - 16, INVALID), (x - proj + 16, INVALID),
                         (x + rows, CUDA), (x - proj, CUDA)):
            out.append((want, _layer_call(**{n: x, "proj": at}), ("proj on " + n, at - x)))
    return out


def test_layer_refuses_outputs_that_share_memory(hidden):  # noqa: F811
    """The residual reads x behind the first rows of y, and the gate the projection."""
    assert not wrong(hidden.apply(_layer_overlap))


def test_a_caches_buffers_are_fixed():
    """The library is given the buffers' addresses once: a buffer put in another's
    place would not be the one that calls use."""
    import torch
    c = ops.QuantCache.empty(8, 2, 64, 32, device="cpu")
    for f in FIELDS:
        kept = getattr(c, f)
        assert getattr(c._c, f) == kept.data_ptr()
        with pytest.raises(AttributeError, match="QuantCache"):
            setattr(c, f, torch.zeros_like(kept))
        assert getattr(c, f) is kept
    with pytest.raises(AttributeError):
        c.rows = 4
    c.weight.copy_(torch.ones(8))      # their contents are the caller's


def test_a_stream_of_another_device_is_refused():
    import torch

    class OnDevice1:
        cuda_stream, device, device_index = 1234, torch.device("cuda", 1), 1
    with pytest.raises(ValueError, match="stream"):
        ops._Launch(0, OnDevice1())


def test_host_numbers_that_do_not_fit_are_refused():
    """A keep_pos of 2^31 as int64 is not -2^31 (which would keep every row)."""
    import torch
    c = ops.QuantCache.empty(8, 2, 32, 32, device="cpu")
    for keep in (np.array([2 ** 31]), torch.tensor([2 ** 31]), [2 ** 31], [1.5], [float("nan")],
                 np.array([-2 ** 31 - 1])):
        with pytest.raises(ValueError, match="keep_pos"):
            ops.qcache_evict(c, [0], [4], [2], keep)
    for bad in ([0.5], np.array([2.0 ** 64])):
        with pytest.raises(ValueError, match="lens"):
            ops.qcache_evict(c, [0], bad, [2], [0])
    for good in ([3], np.array([3.0]), torch.tensor([3], dtype=torch.int32), np.array([3], ">i8")):
        got = ops._host_vec(good, 1, np.int32, "x")
        assert got.tolist() == [3] and got.dtype == np.int32 and got.flags.c_contiguous
    assert ops._host_vec([], 0, np.int64, "x").dtype == np.int64
