"""ctypes binding of libhstu.so (include/hstu.h): argument marshalling only.

Every step of the computation runs in the library's CUDA kernels.  Torch is
used for device memory (outputs, workspaces) and the current stream.  If the
library is missing this module raises at import time -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Sequence

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libhstu.so")
# HSTU_LIB names another build of the same library (the phase-traced one of
# `build --trace`); unset, the in-tree library above is loaded.
LIB_PATH = os.environ.get("HSTU_LIB") or LIB_PATH

HSTU_OK = 0
STATUS = {0: "HSTU_OK", 1: "HSTU_ERR_INVALID_ARG", 2: "HSTU_ERR_UNSUPPORTED",
          3: "HSTU_ERR_WORKSPACE", 4: "HSTU_ERR_CUDA", 5: "HSTU_ERR_DEVICE_TIMEOUT",
          6: "HSTU_ERR_DEVICE"}
F32, BF16 = 0, 1
MASK_CAUSAL, MASK_MFALCON = 0, 1
IMPL = {"auto": 0, "simt": 1}

EXPORTED = [
    "hstu_status_string", "hstu_version", "hstu_attn_workspace_size", "hstu_attn_fwd",
    "hstu_attn_bwd", "hstu_layer_workspace_size", "hstu_layer_fwd", "hstu_debug_buckets",
    "hstu_get_device_error", "hstu_set_wait_limit", "hstu_kernel_launch_count",
    "hstu_attn_fwd_noalloc", "hstu_debug_wait_probe", "hstu_partition_batch",
    "hstu_layer_bwd_workspace_size", "hstu_layer_bwd", "hstu_layer_fwd_keep_proj",
    "hstu_attn_candidates_workspace_size", "hstu_attn_fwd_candidates",
    "hstu_layer_candidates_workspace_size", "hstu_layer_fwd_candidates",
    "hstu_debug_trace_read", "hstu_debug_trace_clear", "hstu_debug_plan",
    "hstu_qcache_append", "hstu_qcache_read", "hstu_qcache_evict_workspace_size",
    "hstu_qcache_evict", "hstu_attn_candidates_qcache_workspace_size",
    "hstu_attn_fwd_candidates_qcache", "hstu_layer_candidates_qcache_workspace_size",
    "hstu_layer_fwd_candidates_qcache",
]


class HstuError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what} failed: {STATUS.get(status, status)}")
        self.status = status


class AttnParams(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("num_heads", ctypes.c_int32), ("d_qk", ctypes.c_int32),
        ("d_v", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
        ("num_pos_buckets", ctypes.c_int32), ("num_time_buckets", ctypes.c_int32),
        ("time_bucket_sub_bits", ctypes.c_int32), ("rab_per_head", ctypes.c_int32),
        ("mask", ctypes.c_int32), ("dtype", ctypes.c_int32), ("impl", ctypes.c_int32),
        ("q_row_stride", ctypes.c_int64), ("k_row_stride", ctypes.c_int64),
        ("v_row_stride", ctypes.c_int64), ("o_row_stride", ctypes.c_int64),
        ("do_row_stride", ctypes.c_int64), ("dq_row_stride", ctypes.c_int64),
        ("dk_row_stride", ctypes.c_int64), ("dv_row_stride", ctypes.c_int64),
        ("alpha", ctypes.c_float), ("silu_scale", ctypes.c_float),
    ]


class LayerParams(ctypes.Structure):
    _fields_ = [("attn", AttnParams), ("d_model", ctypes.c_int32),
                ("residual", ctypes.c_int32), ("ln_eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class _QCacheStruct(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("num_heads", ctypes.c_int32), ("d_qk", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("times", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("weight", ctypes.c_void_p)]


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(f"libhstu.so not found at {path}; build it with "
                           "`python -m hstu_pointwise_attention_b200.build`")
    lib = ctypes.CDLL(path)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
    P, LP = ctypes.POINTER(AttnParams), ctypes.POINTER(LayerParams)
    lib.hstu_status_string.argtypes = [ctypes.c_int]
    lib.hstu_status_string.restype = ctypes.c_char_p
    lib.hstu_version.restype = ctypes.c_char_p
    lib.hstu_attn_workspace_size.argtypes = [P, vp, i32, ctypes.POINTER(sz)]
    lib.hstu_attn_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.hstu_attn_bwd.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                  vp, sz, vp]
    lib.hstu_layer_workspace_size.argtypes = [LP, vp, ctypes.POINTER(sz)]
    lib.hstu_layer_fwd.argtypes = [LP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                   sz, vp]
    lib.hstu_debug_buckets.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.hstu_get_device_error.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_uint32)]
    lib.hstu_set_wait_limit.argtypes = [ctypes.c_uint32]
    lib.hstu_set_wait_limit.restype = None
    lib.hstu_kernel_launch_count.argtypes = []
    lib.hstu_kernel_launch_count.restype = ctypes.c_uint64
    lib.hstu_attn_fwd_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.hstu_attn_fwd_noalloc.restype = ctypes.c_int
    lib.hstu_debug_wait_probe.argtypes = [vp, sz, ctypes.c_uint32, vp]
    lib.hstu_debug_wait_probe.restype = ctypes.c_int
    lib.hstu_layer_bwd_workspace_size.argtypes = [LP, vp, ctypes.POINTER(sz)]
    lib.hstu_layer_bwd.argtypes = [LP] + [vp] * 23 + [sz, vp]
    i64 = ctypes.c_int64
    lib.hstu_layer_fwd_keep_proj.argtypes = [LP] + [vp] * 15 + [sz, vp]
    lib.hstu_attn_candidates_workspace_size.argtypes = [P, vp, vp, ctypes.POINTER(sz)]
    lib.hstu_attn_fwd_candidates.argtypes = [P] + [vp] * 9 + [i64, i64] + [vp] * 4 + [sz, vp]
    lib.hstu_layer_candidates_workspace_size.argtypes = [LP, vp, vp, ctypes.POINTER(sz)]
    lib.hstu_layer_fwd_candidates.argtypes = [LP] + [vp] * 16 + [sz, vp]
    lib.hstu_partition_batch.argtypes = [vp, vp, i32, i32, vp, vp]
    lib.hstu_partition_batch.restype = ctypes.c_int
    lib.hstu_debug_trace_read.argtypes = [i32, vp, sz]
    lib.hstu_debug_trace_read.restype = ctypes.c_int
    lib.hstu_debug_trace_clear.argtypes = [i32]
    lib.hstu_debug_trace_clear.restype = ctypes.c_int
    lib.hstu_debug_plan.argtypes = [P, vp, vp, i32, vp, vp, vp, vp]
    lib.hstu_debug_plan.restype = ctypes.c_int
    f32, QP = ctypes.c_float, ctypes.POINTER(_QCacheStruct)
    lib.hstu_qcache_append.argtypes = [QP, i32, i32] + [vp] * 4 + [i64, vp, i64, vp, vp]
    lib.hstu_qcache_read.argtypes = [QP, i32, i32, vp, vp, vp, i64, vp, i64, vp]
    lib.hstu_qcache_evict_workspace_size.argtypes = [i32, vp, vp, ctypes.POINTER(sz)]
    lib.hstu_qcache_evict.argtypes = [QP, QP, i32] + [vp] * 6 + [sz, vp]
    lib.hstu_attn_candidates_qcache_workspace_size.argtypes = [P, vp, vp, i32,
                                                               ctypes.POINTER(sz)]
    lib.hstu_attn_fwd_candidates_qcache.argtypes = [P, QP] + [vp] * 10 + [i32, f32, vp, vp, sz,
                                                                         vp]
    lib.hstu_layer_candidates_qcache_workspace_size.argtypes = [LP, vp, vp, i32,
                                                                ctypes.POINTER(sz)]
    lib.hstu_layer_fwd_candidates_qcache.argtypes = [LP, QP] + [vp] * 14 + [i32, f32, vp, vp, vp,
                                                                           sz, vp]
    for name in ("hstu_attn_workspace_size", "hstu_attn_fwd", "hstu_attn_bwd",
                 "hstu_layer_workspace_size", "hstu_layer_fwd", "hstu_debug_buckets",
                 "hstu_get_device_error", "hstu_layer_bwd_workspace_size", "hstu_layer_bwd",
                 "hstu_layer_fwd_keep_proj", "hstu_attn_candidates_workspace_size",
                 "hstu_attn_fwd_candidates", "hstu_layer_candidates_workspace_size",
                 "hstu_layer_fwd_candidates", "hstu_qcache_append", "hstu_qcache_read",
                 "hstu_qcache_evict_workspace_size", "hstu_qcache_evict",
                 "hstu_attn_candidates_qcache_workspace_size", "hstu_attn_fwd_candidates_qcache",
                 "hstu_layer_candidates_qcache_workspace_size",
                 "hstu_layer_fwd_candidates_qcache"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


LIB = load()


def _check(rc: int, what: str) -> None:
    if rc != HSTU_OK:
        raise HstuError(rc, what)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _host_i64(a) -> np.ndarray:
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a, dtype=np.int64))


def _host_i32(a) -> Optional[np.ndarray]:
    if a is None:
        return None
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _row_stride(t: torch.Tensor, H: int, d: int, name: str) -> int:
    """t is [T, H, d] (or a [T, H*d] view) with contiguous heads.  Strides that carry no
    meaning are not looked at: an empty tensor's, and in a contiguous one those of
    dimensions of size 1."""
    if t.dim() == 3 and t.shape[1:] == (H, d) and t.is_contiguous():
        return H * d
    if t.dim() in (2, 3) and t.shape[0] == 0 and tuple(t.shape[1:]) in ((H, d), (H * d,)):
        return H * d
    if t.dim() == 3:
        if t.shape[1:] != (H, d) or t.stride()[1:] != (d, 1):
            raise ValueError(f"{name}: expected [T, {H}, {d}] with contiguous heads")
    elif t.dim() == 2:
        if t.shape[1] != H * d or t.stride(1) != 1:
            raise ValueError(f"{name}: expected [T, {H * d}] with unit column stride")
    else:
        raise ValueError(f"{name}: expected 2 or 3 dims")
    return int(t.stride(0)) if t.shape[0] > 1 else H * d


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def make_params(q, k, v, seq_offsets, *, max_seq_len, num_pos_buckets, num_time_buckets,
                time_bucket_sub_bits, alpha=None, silu_scale=None, num_candidates=None,
                rab_per_head=False, impl="auto", out=None, dout=None, dq=None, dk=None,
                dv=None) -> AttnParams:
    H = q.shape[1] if q.dim() == 3 else None
    if H is None:
        raise ValueError("q must be [T, H, d_qk]")
    d_qk, d_v = q.shape[2], v.shape[-1] if v.dim() == 3 else v.shape[1] // H
    off = _host_i64(seq_offsets)
    p = AttnParams()
    p.batch = len(off) - 1
    p.num_heads = H
    p.d_qk, p.d_v = d_qk, d_v
    p.max_seq_len = int(max_seq_len)
    p.num_pos_buckets, p.num_time_buckets = int(num_pos_buckets), int(num_time_buckets)
    p.time_bucket_sub_bits = int(time_bucket_sub_bits)
    p.rab_per_head = int(bool(rab_per_head))
    p.mask = MASK_MFALCON if num_candidates is not None else MASK_CAUSAL
    if q.dtype == torch.float32:
        p.dtype = F32
    elif q.dtype == torch.bfloat16:
        p.dtype = BF16
    else:
        raise ValueError(f"unsupported dtype {q.dtype}")
    for t, name in ((k, "k"), (v, "v")):
        if t.dtype != q.dtype:
            raise ValueError(f"{name} dtype {t.dtype} != q dtype {q.dtype}")
    p.impl = IMPL[impl]
    p.q_row_stride = _row_stride(q, H, d_qk, "q")
    p.k_row_stride = _row_stride(k, H, d_qk, "k")
    p.v_row_stride = _row_stride(v, H, d_v, "v")
    p.o_row_stride = _row_stride(out, H, d_v, "out") if out is not None else H * d_v
    p.do_row_stride = _row_stride(dout, H, d_v, "dout") if dout is not None else H * d_v
    p.dq_row_stride = _row_stride(dq, H, d_qk, "dq") if dq is not None else H * d_qk
    p.dk_row_stride = _row_stride(dk, H, d_qk, "dk") if dk is not None else H * d_qk
    p.dv_row_stride = _row_stride(dv, H, d_v, "dv") if dv is not None else H * d_v
    p.alpha = float(1.0 / math.sqrt(d_qk) if alpha is None else alpha)
    p.silu_scale = float(1.0 / max(1, int(max_seq_len)) if silu_scale is None else silu_scale)
    return p


def attn_workspace_size(p: AttnParams, seq_offsets, is_bwd: bool) -> int:
    off = _host_i64(seq_offsets)
    n = ctypes.c_size_t(0)
    _check(LIB.hstu_attn_workspace_size(ctypes.byref(p), off.ctypes.data, int(is_bwd),
                                        ctypes.byref(n)), "hstu_attn_workspace_size")
    return int(n.value)


def _workspace(nbytes: int, device, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def attn_fwd(q, k, v, seq_offsets, timestamps, rab_pos, rab_time, *, max_seq_len,
             time_bucket_sub_bits, alpha=None, silu_scale=None, num_candidates=None,
             rab_per_head=False, impl="auto", out=None, workspace=None, stream=None):
    """out[T, H, d_v] = HSTU pointwise attention (include/hstu.h)."""
    T, H = q.shape[0], q.shape[1]
    d_v = v.shape[-1] if v.dim() == 3 else v.shape[1] // H
    if out is None:
        out = torch.empty((T, H, d_v), dtype=q.dtype, device=q.device)
    nbp = rab_pos.shape[-1]
    nbt = rab_time.shape[-1]
    p = make_params(q, k, v, seq_offsets, max_seq_len=max_seq_len, num_pos_buckets=nbp,
                    num_time_buckets=nbt, time_bucket_sub_bits=time_bucket_sub_bits, alpha=alpha,
                    silu_scale=silu_scale, num_candidates=num_candidates,
                    rab_per_head=rab_per_head, impl=impl, out=out)
    off = _host_i64(seq_offsets)
    nc = _host_i32(num_candidates)
    ws = _workspace(attn_workspace_size(p, off, False), q.device, workspace)
    _check(LIB.hstu_attn_fwd(ctypes.byref(p), off.ctypes.data,
                             None if nc is None else nc.ctypes.data, _ptr(timestamps), _ptr(q),
                             _ptr(k), _ptr(v), _ptr(rab_pos), _ptr(rab_time), _ptr(out),
                             _ptr(ws), ws.numel(), _stream(stream)), "hstu_attn_fwd")
    return out


def attn_bwd(q, k, v, seq_offsets, timestamps, rab_pos, rab_time, dout, *, max_seq_len,
             time_bucket_sub_bits, alpha=None, silu_scale=None, num_candidates=None,
             rab_per_head=False, impl="auto", dq=None, dk=None, dv=None, drab_pos=None,
             drab_time=None, workspace=None, stream=None):
    """(dq, dk, dv, drab_pos, drab_time); drab_* are accumulated into if given."""
    if dq is None:
        dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if dk is None:
        dk = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    if dv is None:
        dv = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    if drab_pos is None:
        drab_pos = torch.zeros(rab_pos.shape, dtype=torch.float32, device=q.device)
    if drab_time is None:
        drab_time = torch.zeros(rab_time.shape, dtype=torch.float32, device=q.device)
    p = make_params(q, k, v, seq_offsets, max_seq_len=max_seq_len,
                    num_pos_buckets=rab_pos.shape[-1], num_time_buckets=rab_time.shape[-1],
                    time_bucket_sub_bits=time_bucket_sub_bits, alpha=alpha,
                    silu_scale=silu_scale, num_candidates=num_candidates,
                    rab_per_head=rab_per_head, impl=impl, dout=dout, dq=dq, dk=dk, dv=dv)
    off = _host_i64(seq_offsets)
    nc = _host_i32(num_candidates)
    ws = _workspace(attn_workspace_size(p, off, True), q.device, workspace)
    _check(LIB.hstu_attn_bwd(ctypes.byref(p), off.ctypes.data,
                             None if nc is None else nc.ctypes.data, _ptr(timestamps), _ptr(q),
                             _ptr(k), _ptr(v), _ptr(rab_pos), _ptr(rab_time), _ptr(dout),
                             _ptr(dq), _ptr(dk), _ptr(dv), _ptr(drab_pos), _ptr(drab_time),
                             _ptr(ws), ws.numel(), _stream(stream)), "hstu_attn_bwd")
    return dq, dk, dv, drab_pos, drab_time


def _layer_params(x, rab_pos, rab_time, seq_offsets, num_candidates, *, num_heads, d_qk, d_v,
                  max_seq_len, time_bucket_sub_bits, alpha, silu_scale, ln_eps, residual):
    off = _host_i64(seq_offsets)
    nc = _host_i32(num_candidates)
    lp = LayerParams()
    a = lp.attn
    a.batch = len(off) - 1
    a.num_heads, a.d_qk, a.d_v = num_heads, d_qk, d_v
    a.max_seq_len = int(max_seq_len)
    a.num_pos_buckets, a.num_time_buckets = rab_pos.shape[-1], rab_time.shape[-1]
    a.time_bucket_sub_bits = int(time_bucket_sub_bits)
    a.rab_per_head = 0
    a.mask = MASK_MFALCON if nc is not None else MASK_CAUSAL
    a.dtype = BF16
    a.impl = 0
    a.alpha = float(1.0 / math.sqrt(d_qk) if alpha is None else alpha)
    a.silu_scale = float(1.0 / max(1, int(max_seq_len)) if silu_scale is None else silu_scale)
    lp.d_model = x.shape[1]
    lp.residual = int(bool(residual))
    lp.ln_eps = float(ln_eps)
    return lp, off, nc


def layer_fwd(x, w1, b1, ln_gamma, ln_beta, w2, b2, rab_pos, rab_time, seq_offsets, timestamps,
              *, num_heads, d_qk, d_v, max_seq_len, time_bucket_sub_bits, alpha=None,
              silu_scale=None, num_candidates=None, ln_eps=1e-5, residual=True, out=None,
              workspace=None, stream=None):
    """One HSTU layer forward, bf16 (include/hstu.h, hstu_layer_fwd)."""
    T, D = x.shape
    if out is None:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=x.device)
    lp, off, nc = _layer_params(x, rab_pos, rab_time, seq_offsets, num_candidates,
                                num_heads=num_heads, d_qk=d_qk, d_v=d_v, max_seq_len=max_seq_len,
                                time_bucket_sub_bits=time_bucket_sub_bits, alpha=alpha,
                                silu_scale=silu_scale, ln_eps=ln_eps, residual=residual)
    n = ctypes.c_size_t(0)
    _check(LIB.hstu_layer_workspace_size(ctypes.byref(lp), off.ctypes.data, ctypes.byref(n)),
           "hstu_layer_workspace_size")
    ws = _workspace(int(n.value), x.device, workspace)
    _check(LIB.hstu_layer_fwd(ctypes.byref(lp), off.ctypes.data,
                              None if nc is None else nc.ctypes.data, _ptr(timestamps), _ptr(x),
                              _ptr(w1), _ptr(b1), _ptr(ln_gamma), _ptr(ln_beta), _ptr(w2),
                              _ptr(b2), _ptr(rab_pos), _ptr(rab_time), _ptr(out), _ptr(ws),
                              ws.numel(), _stream(stream)), "hstu_layer_fwd")
    return out


def layer_fwd_keep_proj(x, w1, b1, ln_gamma, ln_beta, w2, b2, rab_pos, rab_time, seq_offsets,
                        timestamps, *, num_heads, d_qk, d_v, max_seq_len, time_bucket_sub_bits,
                        alpha=None, silu_scale=None, num_candidates=None, ln_eps=1e-5,
                        residual=True, out=None, proj_out=None, workspace=None, stream=None):
    """hstu_layer_fwd_keep_proj: (y, proj) with proj = [U|V|Q|K] [T, N1] bf16,
    the history K/V cache of the M-FALCON candidate path."""
    T, D = x.shape
    n1 = 2 * num_heads * (d_v + d_qk)
    if out is None:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=x.device)
    if proj_out is None:
        proj_out = torch.empty((T, n1), dtype=torch.bfloat16, device=x.device)
    lp, off, nc = _layer_params(x, rab_pos, rab_time, seq_offsets, num_candidates,
                                num_heads=num_heads, d_qk=d_qk, d_v=d_v, max_seq_len=max_seq_len,
                                time_bucket_sub_bits=time_bucket_sub_bits, alpha=alpha,
                                silu_scale=silu_scale, ln_eps=ln_eps, residual=residual)
    n = ctypes.c_size_t(0)
    _check(LIB.hstu_layer_workspace_size(ctypes.byref(lp), off.ctypes.data, ctypes.byref(n)),
           "hstu_layer_workspace_size")
    ws = _workspace(int(n.value), x.device, workspace)
    _check(LIB.hstu_layer_fwd_keep_proj(
        ctypes.byref(lp), off.ctypes.data, None if nc is None else nc.ctypes.data,
        _ptr(timestamps), _ptr(x), _ptr(w1), _ptr(b1), _ptr(ln_gamma), _ptr(ln_beta), _ptr(w2),
        _ptr(b2), _ptr(rab_pos), _ptr(rab_time), _ptr(out), _ptr(proj_out), _ptr(ws),
        ws.numel(), _stream(stream)), "hstu_layer_fwd_keep_proj")
    return out, proj_out


def attn_fwd_candidates(q, k, v, k_hist, v_hist, hist_offsets, cand_offsets, hist_timestamps,
                        cand_timestamps, rab_pos, rab_time, *, max_seq_len,
                        time_bucket_sub_bits, alpha=None, silu_scale=None, rab_per_head=False,
                        out=None, workspace=None, stream=None):
    """hstu_attn_fwd_candidates: out[Tc, H, d_v] for a candidate micro-batch
    against cached history keys / values k_hist, v_hist [Th, H, d]."""
    Tc, H = q.shape[0], q.shape[1]
    d_v = v.shape[-1] if v.dim() == 3 else v.shape[1] // H
    if out is None:
        out = torch.empty((Tc, H, d_v), dtype=q.dtype, device=q.device)
    hoff = _host_i64(hist_offsets)
    coff = _host_i64(cand_offsets)
    p = make_params(q, k, v, coff, max_seq_len=max_seq_len, num_pos_buckets=rab_pos.shape[-1],
                    num_time_buckets=rab_time.shape[-1],
                    time_bucket_sub_bits=time_bucket_sub_bits, alpha=alpha,
                    silu_scale=silu_scale, rab_per_head=rab_per_head, out=out)
    kh_rs = _row_stride(k_hist, H, q.shape[2], "k_hist")
    vh_rs = _row_stride(v_hist, H, d_v, "v_hist")
    n = ctypes.c_size_t(0)
    _check(LIB.hstu_attn_candidates_workspace_size(ctypes.byref(p), hoff.ctypes.data,
                                                   coff.ctypes.data, ctypes.byref(n)),
           "hstu_attn_candidates_workspace_size")
    ws = _workspace(int(n.value), q.device, workspace)
    _check(LIB.hstu_attn_fwd_candidates(
        ctypes.byref(p), hoff.ctypes.data, coff.ctypes.data, _ptr(hist_timestamps),
        _ptr(cand_timestamps), _ptr(q), _ptr(k), _ptr(v), _ptr(k_hist), _ptr(v_hist), kh_rs,
        vh_rs, _ptr(rab_pos), _ptr(rab_time), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
        "hstu_attn_fwd_candidates")
    return out


def layer_fwd_candidates(x_cand, w1, b1, ln_gamma, ln_beta, w2, b2, rab_pos, rab_time,
                         hist_proj, hist_offsets, cand_offsets, hist_timestamps,
                         cand_timestamps, *, num_heads, d_qk, d_v, max_seq_len,
                         time_bucket_sub_bits, alpha=None, silu_scale=None, ln_eps=1e-5,
                         residual=True, out=None, workspace=None, stream=None):
    """hstu_layer_fwd_candidates: one layer on a candidate micro-batch against
    the history projection kept by layer_fwd_keep_proj."""
    Tc, D = x_cand.shape
    if out is None:
        out = torch.empty((Tc, D), dtype=torch.bfloat16, device=x_cand.device)
    hoff = _host_i64(hist_offsets)
    coff = _host_i64(cand_offsets)
    lp, _, _ = _layer_params(x_cand, rab_pos, rab_time, coff, None, num_heads=num_heads,
                             d_qk=d_qk, d_v=d_v, max_seq_len=max_seq_len,
                             time_bucket_sub_bits=time_bucket_sub_bits, alpha=alpha,
                             silu_scale=silu_scale, ln_eps=ln_eps, residual=residual)
    lp.attn.mask = MASK_MFALCON
    n = ctypes.c_size_t(0)
    _check(LIB.hstu_layer_candidates_workspace_size(ctypes.byref(lp), hoff.ctypes.data,
                                                    coff.ctypes.data, ctypes.byref(n)),
           "hstu_layer_candidates_workspace_size")
    ws = _workspace(int(n.value), x_cand.device, workspace)
    _check(LIB.hstu_layer_fwd_candidates(
        ctypes.byref(lp), hoff.ctypes.data, coff.ctypes.data, _ptr(hist_timestamps),
        _ptr(cand_timestamps), _ptr(x_cand), _ptr(w1), _ptr(b1), _ptr(ln_gamma), _ptr(ln_beta),
        _ptr(w2), _ptr(b2), _ptr(rab_pos), _ptr(rab_time), _ptr(hist_proj), _ptr(out),
        _ptr(ws), ws.numel(), _stream(stream)), "hstu_layer_fwd_candidates")
    return out


class QuantCache:
    """The buffers of one layer's 4-bit history cache (include/hstu.h,
    hstu_qcache_t): k_codes, v_codes uint8 [H, rows, d / 2]; k_scales, v_scales
    int16 [H, rows, d / 32]; times int64, pos int32, weight float32 [rows]
    (weight may be None where no call updates or reads it).  Contiguous, on one
    CUDA device, and the same for the object's life (their contents may change).
    ``QuantCache.empty`` allocates them."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales, times, pos, weight=None):
        H, rows, half_k = k_codes.shape
        half_v = v_codes.shape[2]
        want = [("k_codes", k_codes, (torch.uint8,), (H, rows, half_k)),
                ("k_scales", k_scales, (torch.int16, torch.uint16), (H, rows, half_k // 16)),
                ("v_codes", v_codes, (torch.uint8,), (H, rows, half_v)),
                ("v_scales", v_scales, (torch.int16, torch.uint16), (H, rows, half_v // 16)),
                ("times", times, (torch.int64,), (rows,)), ("pos", pos, (torch.int32,), (rows,)),
                ("weight", weight, (torch.float32,), (rows,))]
        for name, t, dtypes, shape in want:
            if t is None and name == "weight":
                continue
            if t.dtype not in dtypes or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name}: expected contiguous {dtypes[0]} {list(shape)}, got "
                                 f"{t.dtype} {list(t.shape)}")
            if t.device != k_codes.device:
                raise ValueError(f"{name} is on {t.device}, k_codes on {k_codes.device}")
        if half_k % 16 or half_v % 16:
            raise ValueError("head sizes must be multiples of 32")
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = (k_codes, k_scales, v_codes,
                                                                     v_scales)
        self.times, self.pos, self.weight = times, pos, weight
        self.rows, self.num_heads, self.d_qk, self.d_v = rows, H, 2 * half_k, 2 * half_v
        self.device, self._index = k_codes.device, k_codes.get_device()
        self._c = _QCacheStruct(rows, H, self.d_qk, self.d_v, 0, _ptr(k_codes), _ptr(k_scales),
                                _ptr(v_codes), _ptr(v_scales), _ptr(times), _ptr(pos),
                                _ptr(weight))

    def __setattr__(self, name, value):
        if name in self.__dict__:      # the library's copy would keep the old address
            raise AttributeError(f"QuantCache.{name} is fixed; make a new QuantCache")
        super().__setattr__(name, value)

    @classmethod
    def empty(cls, rows, num_heads, d_qk, d_v, device="cuda"):
        z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
        return cls(z((num_heads, rows, d_qk // 2), torch.uint8),
                   z((num_heads, rows, d_qk // 32), torch.int16),
                   z((num_heads, rows, d_v // 2), torch.uint8),
                   z((num_heads, rows, d_v // 32), torch.int16), z((rows,), torch.int64),
                   z((rows,), torch.int32), z((rows,), torch.float32))


def _cuda_index(t, *others) -> int:
    """Index of the CUDA device that t and the others (None aside) live on."""
    i = t.get_device()
    if i < 0:
        raise ValueError(f"expected CUDA tensors, got {t.device}")
    for o in others:
        if o is not None and o.get_device() != i:
            raise ValueError(f"tensors on {o.device} and {t.device}")
    return i


class _Launch:
    """Makes the tensors' device current for a call, and the call's stream the
    one its own allocations belong to (a workspace is then reused only behind
    the work that uses it).  Entering gives the raw stream."""
    __slots__ = ("_ctx", "_index")

    def __init__(self, index, stream):
        self._index = index
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream),
                                                   device=torch.device("cuda", index))
            elif stream.device_index != index:
                raise ValueError(f"the stream belongs to {stream.device}, the tensors to "
                                 f"cuda:{index}")
            self._ctx = torch.cuda.stream(stream)
        else:
            self._ctx = None if index == torch.cuda.current_device() else \
                torch.cuda.device(index)

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()
        # the raw stream without a Stream object around it (a microsecond per call)
        return torch._C._cuda_getCurrentRawStream(self._index)

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)
        return False


def _host_vec(a, n, dtype, name):
    if not (type(a) is np.ndarray and a.dtype == dtype and a.flags.c_contiguous):
        raw = a.detach().cpu().numpy() if isinstance(a, torch.Tensor) else np.asarray(a)
        with np.errstate(invalid="ignore"):
            a = np.ascontiguousarray(raw.astype(dtype))
        if not np.array_equal(a, raw):
            raise ValueError(f"{name}: expected whole numbers that fit {np.dtype(dtype)}")
    if a.shape != (n,):
        raise ValueError(f"{name}: expected {n} entries, got shape {a.shape}")
    return a


def _np_ptr(a) -> int:
    """Address of a host array's data (ndarray.ctypes builds an object per use,
    several microseconds for the arrays of one call)."""
    try:
        return ctypes.addressof(ctypes.c_char.from_buffer(a))
    except (TypeError, ValueError, BufferError):    # read-only or empty
        return a.ctypes.data


def _host_offsets(a):
    a = _host_vec(a, len(a), np.int64, "offsets")
    if len(a) < 1:
        raise ValueError("offsets: expected batch + 1 entries")
    return a


def _typed(t, dtype, name):
    if t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype}, got {t.dtype}")
    return t


def _act_dtype(t, name):
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise ValueError(f"{name}: unsupported dtype {t.dtype}")


def qcache_append(cache, k, v, timestamps, tok_offsets, rows, pos, *, stream=None):
    """hstu_qcache_append: quantise new tokens' keys and values [T, H, d] into
    the cache; sequence b's tokens tok_offsets[b]..tok_offsets[b + 1] go to rows
    rows[b].. at positions pos[b]..."""
    off = _host_offsets(tok_offsets)
    B = len(off) - 1
    rows, pos = _host_vec(rows, B, np.int64, "rows"), _host_vec(pos, B, np.int32, "pos")
    dt = _act_dtype(k, "k")
    if v.dtype != k.dtype:
        raise ValueError(f"v dtype {v.dtype} != k dtype {k.dtype}")
    T = int(off[-1]) if B else 0
    if k.shape[0] < T or v.shape[0] < T or timestamps.shape[0] < T:
        raise ValueError(f"k, v and timestamps need {T} tokens")
    k_rs = _row_stride(k, cache.num_heads, cache.d_qk, "k")
    v_rs = _row_stride(v, cache.num_heads, cache.d_v, "v")
    _typed(timestamps, torch.int64, "timestamps")
    with _Launch(_cuda_index(cache.k_codes, k, v, timestamps), stream) as st:
        _check(LIB.hstu_qcache_append(ctypes.byref(cache._c), dt, B, _np_ptr(off),
                                      _np_ptr(rows), _np_ptr(pos), _ptr(k), k_rs, _ptr(v),
                                      v_rs, _ptr(timestamps), st), "hstu_qcache_append")


def qcache_read(cache, rows, lens, *, dtype=torch.bfloat16, k=None, v=None, stream=None):
    """hstu_qcache_read: (k, v) [sum lens, H, d], the values that rows stand for."""
    lens = _host_vec(lens, len(lens), np.int64, "lens")
    rows = _host_vec(rows, len(lens), np.int64, "rows")
    T = sum(lens.tolist())
    with _Launch(_cuda_index(cache.k_codes, k, v), stream) as st:
        if k is None:
            k = torch.empty((T, cache.num_heads, cache.d_qk), dtype=dtype, device=cache.device)
        if v is None:
            v = torch.empty((T, cache.num_heads, cache.d_v), dtype=dtype, device=cache.device)
        if k.dtype != v.dtype or k.shape[0] < T or v.shape[0] < T:
            raise ValueError(f"k and v must share a dtype and hold {T} tokens")
        k_rs = _row_stride(k, cache.num_heads, cache.d_qk, "k")
        v_rs = _row_stride(v, cache.num_heads, cache.d_v, "v")
        _check(LIB.hstu_qcache_read(ctypes.byref(cache._c), _act_dtype(k, "k"), len(lens),
                                    _np_ptr(rows), _np_ptr(lens), _ptr(k), k_rs, _ptr(v),
                                    v_rs, st), "hstu_qcache_read")
    return k, v


def qcache_evict(cache, rows, lens, budgets, keep_pos, *, dst=None, dst_rows=None,
                 workspace=None, stream=None):
    """hstu_qcache_evict: keep each sequence's budgets[b] most used rows, in
    place or (dst, dst_rows) in another cache.  Returns the new lengths."""
    lens = _host_vec(lens, len(lens), np.int64, "lens")
    B = len(lens)
    rows = _host_vec(rows, B, np.int64, "rows")
    budgets = _host_vec(budgets, B, np.int64, "budgets")
    keep_pos = _host_vec(keep_pos, B, np.int32, "keep_pos")
    if (dst is None) != (dst_rows is None):
        raise ValueError("dst and dst_rows go together")
    if cache.weight is None or (dst is not None and dst.weight is None):
        raise ValueError("evicting needs caches with weights")
    if dst is not None and dst.device != cache.device:
        raise ValueError(f"caches on {cache.device} and {dst.device}")
    to = cache if dst is None else dst
    to_rows = rows if dst is None else _host_vec(dst_rows, B, np.int64, "dst_rows")
    n = ctypes.c_size_t(0)
    _check(LIB.hstu_qcache_evict_workspace_size(B, _np_ptr(lens), _np_ptr(budgets),
                                                ctypes.byref(n)),
           "hstu_qcache_evict_workspace_size")
    with _Launch(_cuda_index(cache.k_codes, workspace), stream) as st:
        ws = _workspace(int(n.value), cache.device, workspace)
        _check(LIB.hstu_qcache_evict(
            ctypes.byref(cache._c), ctypes.byref(to._c), B, _np_ptr(rows), _np_ptr(lens),
            _np_ptr(budgets), _np_ptr(keep_pos), _np_ptr(to_rows), _ptr(ws),
            ws.numel() * ws.element_size(), st), "hstu_qcache_evict")
    return np.minimum(lens, budgets)


def _check_cache_heads(cache, H, d_qk, d_v):
    if (cache.num_heads, cache.d_qk, cache.d_v) != (H, d_qk, d_v):
        raise ValueError(f"the cache holds {cache.num_heads} heads of {cache.d_qk} / "
                         f"{cache.d_v}, the call {H} of {d_qk} / {d_v}")


def attn_fwd_candidates_qcache(q, k, v, cache, cache_rows, cache_lens, cand_offsets, cand_pos,
                               cand_timestamps, rab_pos, rab_time, *, max_seq_len,
                               time_bucket_sub_bits, alpha=None, silu_scale=None,
                               rab_per_head=False, weight_decay=None, impl="auto", out=None,
                               workspace=None, stream=None):
    """hstu_attn_fwd_candidates_qcache: out[Tc, H, d_v] for candidates against
    the 4-bit cache.  weight_decay: None leaves cache.weight alone; a number
    updates it (weight <- weight_decay weight + this call's weights)."""
    if q.dim() != 3:
        raise ValueError("q must be [Tc, H, d_qk]")
    Tc, H = q.shape[0], q.shape[1]
    d_v = v.shape[-1] if v.dim() == 3 else v.shape[1] // H
    dt = _act_dtype(q, "q")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError(f"q, k, v must share a dtype, got {q.dtype}, {k.dtype}, {v.dtype}")
    coff = _host_offsets(cand_offsets)
    B = len(coff) - 1
    rows = _host_vec(cache_rows, B, np.int64, "cache_rows")
    lens = _host_vec(cache_lens, B, np.int64, "cache_lens")
    pos = _host_vec(cand_pos, B, np.int32, "cand_pos")
    _check_cache_heads(cache, H, q.shape[2], d_v)
    n_c = int(coff[-1]) if B else 0
    if min(Tc, k.shape[0], v.shape[0], cand_timestamps.shape[0]) < n_c:
        raise ValueError(f"q, k, v and cand_timestamps need {n_c} candidates")
    if weight_decay is not None and cache.weight is None:
        raise ValueError("weight_decay needs a cache with weights")
    _typed(cand_timestamps, torch.int64, "cand_timestamps")
    for t, name in ((rab_pos, "rab_pos"), (rab_time, "rab_time")):
        _typed(t, torch.float32, name)
        if tuple(t.shape[:-1]) != ((H,) if rab_per_head else ()):
            raise ValueError(f"{name}: unexpected shape {list(t.shape)}")
    with _Launch(_cuda_index(cache.k_codes, q, k, v, cand_timestamps, rab_pos, rab_time, out,
                             workspace), stream) as st:
        if out is None:
            out = torch.empty((Tc, H, d_v), dtype=q.dtype, device=q.device)
        if out.shape[0] < n_c or out.dtype != q.dtype:
            raise ValueError(f"out must hold {n_c} candidates of {q.dtype}")
        d_qk, msl = q.shape[2], int(max_seq_len)
        p = AttnParams(B, H, d_qk, d_v, msl, rab_pos.shape[-1], rab_time.shape[-1],
                       int(time_bucket_sub_bits), int(bool(rab_per_head)), MASK_CAUSAL, dt,
                       IMPL[impl], _row_stride(q, H, d_qk, "q"), _row_stride(k, H, d_qk, "k"),
                       _row_stride(v, H, d_v, "v"), _row_stride(out, H, d_v, "out"), 0, 0, 0, 0,
                       1.0 / math.sqrt(d_qk) if alpha is None else alpha,
                       1.0 / max(1, msl) if silu_scale is None else silu_scale)
        upd, decay = int(weight_decay is not None), float(weight_decay or 0.0)
        n = ctypes.c_size_t(0)
        pp, lens_p, coff_p = ctypes.byref(p), _np_ptr(lens), _np_ptr(coff)
        _check(LIB.hstu_attn_candidates_qcache_workspace_size(
            pp, lens_p, coff_p, upd, ctypes.byref(n)),
            "hstu_attn_candidates_qcache_workspace_size")
        ws = _workspace(int(n.value), q.device, workspace)
        _check(LIB.hstu_attn_fwd_candidates_qcache(
            pp, ctypes.byref(cache._c), _np_ptr(rows), lens_p, coff_p, _np_ptr(pos),
            _ptr(cand_timestamps), _ptr(q), _ptr(k), _ptr(v),
            _ptr(rab_pos), _ptr(rab_time), upd, decay, _ptr(out), _ptr(ws),
            ws.numel() * ws.element_size(), st), "hstu_attn_fwd_candidates_qcache")
    return out


def layer_fwd_candidates_qcache(x_cand, w1, b1, ln_gamma, ln_beta, w2, b2, rab_pos, rab_time,
                                cache, cache_rows, cache_lens, cand_offsets, cand_pos,
                                cand_timestamps, *, num_heads, d_qk, d_v, max_seq_len,
                                time_bucket_sub_bits, alpha=None, silu_scale=None, ln_eps=1e-5,
                                residual=True, weight_decay=None, out=None, proj_out=None,
                                workspace=None, stream=None):
    """hstu_layer_fwd_candidates_qcache: one layer on candidates against the
    4-bit cache of its history.  proj_out [Tc, N1] bf16 (optional) receives the
    candidates' projection [U|V|Q|K]."""
    Tc, D = x_cand.shape
    H, F = num_heads, num_heads * d_v
    n1 = 2 * (F + H * d_qk)
    coff = _host_offsets(cand_offsets)
    B = len(coff) - 1
    rows = _host_vec(cache_rows, B, np.int64, "cache_rows")
    lens = _host_vec(cache_lens, B, np.int64, "cache_lens")
    pos = _host_vec(cand_pos, B, np.int32, "cand_pos")
    _check_cache_heads(cache, H, d_qk, d_v)
    n_c = int(coff[-1]) if B else 0
    bf, f32 = torch.bfloat16, torch.float32
    want = [("x_cand", x_cand, bf, (Tc, D)), ("w1", w1, bf, (n1, D)), ("b1", b1, f32, (n1,)),
            ("ln_gamma", ln_gamma, f32, (F,)), ("ln_beta", ln_beta, f32, (F,)),
            ("w2", w2, bf, (D, F)), ("b2", b2, f32, (D,)),
            ("rab_pos", rab_pos, f32, tuple(rab_pos.shape[-1:])),
            ("rab_time", rab_time, f32, tuple(rab_time.shape[-1:])), ("out", out, bf, (Tc, D)),
            ("proj_out", proj_out, bf, (Tc, n1))]
    for name, t, dt, shape in want:
        if t is not None and (t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous()):
            raise ValueError(f"{name}: expected contiguous {dt} {list(shape)}, got {t.dtype} "
                             f"{list(t.shape)}")
    if min(Tc, cand_timestamps.shape[0]) < n_c:
        raise ValueError(f"x_cand and cand_timestamps need {n_c} candidates")
    if weight_decay is not None and cache.weight is None:
        raise ValueError("weight_decay needs a cache with weights")
    _typed(cand_timestamps, torch.int64, "cand_timestamps")
    with _Launch(_cuda_index(cache.k_codes, x_cand, w1, b1, ln_gamma, ln_beta, w2, b2, rab_pos,
                             rab_time, cand_timestamps, out, proj_out, workspace),
                 stream) as st:
        if out is None:
            out = torch.empty((Tc, D), dtype=bf, device=x_cand.device)
        lp, _, _ = _layer_params(x_cand, rab_pos, rab_time, coff, None, num_heads=H, d_qk=d_qk,
                                 d_v=d_v, max_seq_len=max_seq_len,
                                 time_bucket_sub_bits=time_bucket_sub_bits, alpha=alpha,
                                 silu_scale=silu_scale, ln_eps=ln_eps, residual=residual)
        upd, decay = int(weight_decay is not None), float(weight_decay or 0.0)
        n = ctypes.c_size_t(0)
        _check(LIB.hstu_layer_candidates_qcache_workspace_size(
            ctypes.byref(lp), _np_ptr(lens), _np_ptr(coff), upd, ctypes.byref(n)),
            "hstu_layer_candidates_qcache_workspace_size")
        ws = _workspace(int(n.value), x_cand.device, workspace)
        _check(LIB.hstu_layer_fwd_candidates_qcache(
            ctypes.byref(lp), ctypes.byref(cache._c), _np_ptr(rows), _np_ptr(lens),
            _np_ptr(coff), _np_ptr(pos), _ptr(cand_timestamps), _ptr(x_cand), _ptr(w1),
            _ptr(b1), _ptr(ln_gamma), _ptr(ln_beta), _ptr(w2), _ptr(b2), _ptr(rab_pos),
            _ptr(rab_time), upd, decay, _ptr(out), _ptr(proj_out), _ptr(ws),
            ws.numel() * ws.element_size(), st), "hstu_layer_fwd_candidates_qcache")
    return out


def layer_bwd(x, w1, b1, ln_gamma, ln_beta, w2, b2, rab_pos, rab_time, seq_offsets, timestamps,
              dy, *, num_heads, d_qk, d_v, max_seq_len, time_bucket_sub_bits, alpha=None,
              silu_scale=None, num_candidates=None, ln_eps=1e-5, residual=True, dx=None,
              grads=None, workspace=None, stream=None):
    """One HSTU layer backward (include/hstu.h, hstu_layer_bwd).

    Returns (dx, grads) with grads a dict of float32 tensors dw1, db1,
    dgamma, dbeta, dw2, db2, drab_pos, drab_time; pass ``grads`` to
    accumulate into existing ones (the library adds to them)."""
    T, D = x.shape
    dev = x.device
    if dx is None:
        dx = torch.empty((T, D), dtype=torch.bfloat16, device=dev)
    if grads is None:
        z = lambda t: torch.zeros(t.shape, dtype=torch.float32, device=dev)
        grads = dict(dw1=z(w1), db1=z(b1), dgamma=z(ln_gamma), dbeta=z(ln_beta), dw2=z(w2),
                     db2=z(b2), drab_pos=z(rab_pos), drab_time=z(rab_time))
    lp, off, nc = _layer_params(x, rab_pos, rab_time, seq_offsets, num_candidates,
                                num_heads=num_heads, d_qk=d_qk, d_v=d_v, max_seq_len=max_seq_len,
                                time_bucket_sub_bits=time_bucket_sub_bits, alpha=alpha,
                                silu_scale=silu_scale, ln_eps=ln_eps, residual=residual)
    n = ctypes.c_size_t(0)
    _check(LIB.hstu_layer_bwd_workspace_size(ctypes.byref(lp), off.ctypes.data,
                                             ctypes.byref(n)), "hstu_layer_bwd_workspace_size")
    ws = _workspace(int(n.value), dev, workspace)
    g = grads
    _check(LIB.hstu_layer_bwd(ctypes.byref(lp), off.ctypes.data,
                              None if nc is None else nc.ctypes.data, _ptr(timestamps), _ptr(x),
                              _ptr(w1), _ptr(b1), _ptr(ln_gamma), _ptr(ln_beta), _ptr(w2),
                              _ptr(b2), _ptr(rab_pos), _ptr(rab_time), _ptr(dy), _ptr(dx),
                              _ptr(g["dw1"]), _ptr(g["db1"]), _ptr(g["dgamma"]),
                              _ptr(g["dbeta"]), _ptr(g["dw2"]), _ptr(g["db2"]),
                              _ptr(g["drab_pos"]), _ptr(g["drab_time"]), _ptr(ws), ws.numel(),
                              _stream(stream)), "hstu_layer_bwd")
    return dx, grads


def debug_buckets(seq_offsets, timestamps, *, num_heads, d_qk, d_v, max_seq_len,
                  num_pos_buckets, num_time_buckets, time_bucket_sub_bits,
                  num_candidates=None, stream=None):
    """(bp, bt, bt_fast) int32 device tensors, dense L x L blocks per sequence."""
    off = _host_i64(seq_offsets)
    L = np.diff(off)
    n = int((L.astype(np.int64) ** 2).sum())
    dev = timestamps.device
    dummy = torch.empty((1, num_heads, d_qk), dtype=torch.bfloat16, device=dev)
    dummy_v = torch.empty((1, num_heads, d_v), dtype=torch.bfloat16, device=dev)
    p = make_params(dummy, dummy, dummy_v, off, max_seq_len=max_seq_len,
                    num_pos_buckets=num_pos_buckets, num_time_buckets=num_time_buckets,
                    time_bucket_sub_bits=time_bucket_sub_bits, num_candidates=num_candidates)
    nc = _host_i32(num_candidates)
    ws = _workspace(attn_workspace_size(p, off, False), dev, None)
    bp = torch.empty(max(n, 1), dtype=torch.int32, device=dev)
    bt = torch.empty(max(n, 1), dtype=torch.int32, device=dev)
    btf = torch.empty(max(n, 1), dtype=torch.int32, device=dev)
    _check(LIB.hstu_debug_buckets(ctypes.byref(p), off.ctypes.data,
                                  None if nc is None else nc.ctypes.data, _ptr(timestamps),
                                  _ptr(bp), _ptr(bt), _ptr(btf), _ptr(ws), ws.numel(),
                                  _stream(stream)), "hstu_debug_buckets")
    return bp[:n], bt[:n], btf[:n]


def get_device_error(workspace: torch.Tensor, stream=None):
    detail = ctypes.c_uint32(0)
    rc = LIB.hstu_get_device_error(_ptr(workspace), _stream(stream), ctypes.byref(detail))
    return rc, int(detail.value)


def debug_wait_probe(workspace: torch.Tensor, limit_us: int, stream=None) -> int:
    """hstu_debug_wait_probe: a device wait that runs out after limit_us."""
    return int(LIB.hstu_debug_wait_probe(_ptr(workspace), workspace.numel() *
                                         workspace.element_size(), int(limit_us),
                                         _stream(stream)))


def set_wait_limit(microseconds: int) -> None:
    LIB.hstu_set_wait_limit(int(microseconds))


def attn_fwd_noalloc(q, k, v, seq_offsets, timestamps, rab_pos, rab_time, *, max_seq_len,
                     time_bucket_sub_bits, alpha=None, silu_scale=None, num_candidates=None,
                     rab_per_head=False, impl="auto", out=None, stream=None):
    """hstu_attn_fwd_noalloc: the forward without a workspace, for callers that
    cannot allocate device memory; its scratch is a fixed device array inside
    the library (see include/hstu.h).  `out` must be given by such callers."""
    T, H = q.shape[0], q.shape[1]
    d_v = v.shape[-1] if v.dim() == 3 else v.shape[1] // H
    if out is None:
        out = torch.empty((T, H, d_v), dtype=q.dtype, device=q.device)
    p = make_params(q, k, v, seq_offsets, max_seq_len=max_seq_len,
                    num_pos_buckets=rab_pos.shape[-1], num_time_buckets=rab_time.shape[-1],
                    time_bucket_sub_bits=time_bucket_sub_bits, alpha=alpha,
                    silu_scale=silu_scale, num_candidates=num_candidates,
                    rab_per_head=rab_per_head, impl=impl, out=out)
    off = _host_i64(seq_offsets)
    nc = _host_i32(num_candidates)
    _check(LIB.hstu_attn_fwd_noalloc(ctypes.byref(p), off.ctypes.data,
                                     None if nc is None else nc.ctypes.data, _ptr(timestamps),
                                     _ptr(q), _ptr(k), _ptr(v), _ptr(rab_pos), _ptr(rab_time),
                                     _ptr(out), _stream(stream)), "hstu_attn_fwd_noalloc")
    return out


def partition_batch(seq_offsets, world: int, num_candidates=None):
    """hstu_partition_batch: (rank_of_seq int32 [B], pairs_per_rank int64 [world])."""
    off = _host_i64(seq_offsets)
    nc = _host_i32(num_candidates)
    B = len(off) - 1
    rank_of = np.zeros(max(B, 1), np.int32)
    pairs = np.zeros(max(int(world), 1), np.int64)
    _check(LIB.hstu_partition_batch(off.ctypes.data, None if nc is None else nc.ctypes.data,
                                    int(B), int(world), rank_of.ctypes.data, pairs.ctypes.data),
           "hstu_partition_batch")
    return rank_of[:B], pairs[:int(world)]


def version() -> str:
    return LIB.hstu_version().decode()


def launch_count() -> int:
    """Kernels the library has launched in this process."""
    return int(LIB.hstu_kernel_launch_count())


# Phase traces of the tensor-core kernels (library built with `build --trace`):
# three CTAs x one recorder per warp x entries (code << 56 | ordinal << 40 | clock).
TRACE_SHAPE = (3, 20, 1024)
TRACE_KERNEL = {"bwd": 0, "fwd": 1}


def trace_clear(kernel: str = "bwd") -> None:
    _check(LIB.hstu_debug_trace_clear(TRACE_KERNEL[kernel]), "hstu_debug_trace_clear")


def trace_read(kernel: str = "bwd") -> np.ndarray:
    buf = np.zeros(TRACE_SHAPE, dtype=np.uint64)
    _check(LIB.hstu_debug_trace_read(TRACE_KERNEL[kernel], buf.ctypes.data, buf.nbytes),
           "hstu_debug_trace_read")
    return buf


def debug_plan(p: "AttnParams", seq_offsets, num_candidates=None):
    """(forward items, backward items) as int32 [n, 4] arrays (include/hstu.h,
    hstu_debug_plan); host only."""
    off = _host_i64(seq_offsets)
    nc = _host_i32(num_candidates)
    nf, nb = ctypes.c_int32(0), ctypes.c_int32(0)
    cap = 16
    while True:
        fi = np.zeros((cap, 4), dtype=np.int32)
        bi = np.zeros((cap, 4), dtype=np.int32)
        rc = LIB.hstu_debug_plan(ctypes.byref(p), off.ctypes.data,
                                 None if nc is None else nc.ctypes.data, cap, fi.ctypes.data,
                                 ctypes.byref(nf), bi.ctypes.data, ctypes.byref(nb))
        if rc == HSTU_OK:
            return fi[:nf.value].copy(), bi[:nb.value].copy()
        if nf.value <= cap and nb.value <= cap:
            _check(rc, "hstu_debug_plan")
        cap = max(nf.value, nb.value)
