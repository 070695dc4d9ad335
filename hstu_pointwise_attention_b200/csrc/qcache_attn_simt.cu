// qcache_attn_simt.cu -- candidates against the 4-bit history cache on the
// CUDA cores (any head size, float32 or bf16), and the summing pass of both
// attention kernels.
//
//   out_i = c (sum_j SiLU(x_ij) v_j + SiLU(x_ii) v_i),
//   x_ij = alpha <q_i, k_j> + rab_pos[P_b - pos_j] + rab_time[tb(t_i - t_j)]
//   w_j  <- decay w_j + c sum_{i, h} |SiLU(x_ij)|
//
// One CTA = 16 candidates of one (sequence, head) and a range of keys, 64 keys
// at a time: their rows are decoded to float32 in shared memory, each thread
// makes the weights of one key for 8 candidates, then sums one or two output
// columns over the 64 keys (with at most 64 columns, over every other key).  Bound
// by shared-memory reads: 9 16-byte reads per 32 multiply-adds in the first step,
// 5 per 16 in the second.  32 histories of 64 to 1,024 events, 1 to 24 candidates
// each, 4 heads of 64, float32: 25 us and 5 more to sum, most of it the latency of
// a CTA's few steps (issue slots 25 % busy).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qcache_attn.cuh"

namespace hstu {
namespace qc_simt {

constexpr int kThreads = 128;
constexpr int kQ = kQcSimtQueries;   // candidates per CTA
constexpr int kKeys = 64;            // keys per step
constexpr int kPerThread = kQ / (kThreads / kKeys);
constexpr int kPPitch = kQ + 4;      // P [kKeys][kPPitch]: 8 keys' rows in 8 bank groups

// Shared memory in floats: q [kQ][d_qk], k [kKeys][d_qk + 4], v [kKeys][d_v], P.
__host__ __device__ constexpr size_t smem_floats(int d_qk, int d_v) {
  return size_t(kQ) * d_qk + size_t(kKeys) * (d_qk + 4) + size_t(kKeys) * d_v + kKeys * kPPitch;
}

__device__ __forceinline__ float silu_exact(float x) { return x / (1.0f + expf(-x)); }

// Rows [0, n) of codes to float32 rows of `pitch`, rows [n, kKeys) to zeros.
__device__ __forceinline__ void decode_rows(float *dst, int pitch, const uint32_t *codes,
                                            const uint16_t *scales, int64_t at, int d, int n) {
  const int words = d >> 3;
  for (int x = threadIdx.x; x < kKeys * words; x += kThreads) {
    const int r = x / words, w = x - r * words;
    uint32_t code = 0, par = 0;
    if (r < n) {
      code = codes[(at + r) * words + w];
      par = scales[(at + r) * (d >> 5) + (w >> 2)];
    }
    const float s = q4_scale(par);
    // 2^23 + q as a float is 0x4B000000 | q: less 2^23 + z leaves q - z
    const float z = 8388608.0f + float(par & 15u);
    float o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      o[e] = s * (__uint_as_float(0x4B000000u | uint32_t(q4_code(code, e))) - z);
    float4 *p = reinterpret_cast<float4 *>(dst + r * pitch + 8 * w);
    p[0] = make_float4(o[0], o[1], o[2], o[3]);
    p[1] = make_float4(o[4], o[5], o[6], o[7]);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    attn_kernel(const __grid_constant__ QcAttnParams p) {
  extern __shared__ float4 sm4[];
  const QCacheView &c = p.cache;
  const int H = c.heads, dq = c.d_qk, dv = c.d_v;
  const int item = int(blockIdx.x) / H, h = int(blockIdx.x) - item * H;
  const int tid = threadIdx.x;
  if (p.clear_err && blockIdx.x == 0 && tid < 4) p.wait.err[tid] = 0;
  const QcItem it = qc_item(p, item);
  const QcAttnSeq &sq = p.seqs[it.seq];
  const int i0 = it.qtile * kQ, nq = min(kQ, sq.n - i0);
  float *sq_q = reinterpret_cast<float *>(sm4), *sk = sq_q + kQ * dq, *sv = sk + kKeys * (dq + 4),
        *sp = sv + kKeys * dv;
  __shared__ int64_t s_t[kQ];
  const float *rp = p.rab_p + (p.rab_per_head ? int64_t(h) * p.nb_p : 0);
  const float *rt = p.rab_t + (p.rab_per_head ? int64_t(h) * p.nb_t : 0);

  const T *q = static_cast<const T *>(p.q);
  for (int x = tid; x < kQ * dq; x += kThreads) {
    const int i = x / dq, e = x - i * dq;
    sq_q[x] = i < nq ? qc_float<T>(q[(sq.q0 + i0 + i) * p.q_rs + int64_t(h) * dq + e]) : 0.f;
  }
  if (tid < kQ) s_t[tid] = tid < nq ? p.cand_ts[sq.q0 + i0 + tid] : 0;

  float acc[2][kQ];
#pragma unroll
  for (int a = 0; a < 2; ++a)
#pragma unroll
    for (int i = 0; i < kQ; ++i) acc[a][i] = 0.f;

  const int kj = tid & (kKeys - 1), kg = tid / kKeys;   // key and candidate group of step 1
  const bool paired = dv <= 64;                         // step 2: two threads per column
  const int e0 = paired ? tid & 63 : tid;
  const int32_t j_end = min(it.t1 * kQcKeyTile, sq.len);
  for (int32_t jb = it.t0 * kQcKeyTile; jb < j_end; jb += kKeys) {
    const int nk = min(kKeys, j_end - jb);
    __syncthreads();
    const int64_t at0 = int64_t(h) * c.rows + sq.row + jb;
    decode_rows(sk, dq + 4, c.k_codes, c.k_scales, at0, dq, nk);
    decode_rows(sv, dv, c.v_codes, c.v_scales, at0, dv, nk);
    const bool key_ok = kj < nk;
    const int64_t row = sq.row + jb + (key_ok ? kj : 0);
    const float bp = qc_bias(rp[pos_bucket(int64_t(sq.pos) - c.pos[row], p.nb_p)]);
    const int64_t tk = c.times[row];
    __syncthreads();
    if (kg * kPerThread < nq) {
      float dot[kPerThread];
#pragma unroll
      for (int u = 0; u < kPerThread; ++u) dot[u] = 0.f;
      const float *kr = sk + kj * (dq + 4), *qr = sq_q + kg * kPerThread * dq;
      for (int e = 0; e < dq; e += 4) {
        const float4 kv = *reinterpret_cast<const float4 *>(kr + e);
#pragma unroll
        for (int u = 0; u < kPerThread; ++u) {
          const float4 qv = *reinterpret_cast<const float4 *>(qr + u * dq + e);
          dot[u] = fmaf(qv.x, kv.x, dot[u]);
          dot[u] = fmaf(qv.y, kv.y, dot[u]);
          dot[u] = fmaf(qv.z, kv.z, dot[u]);
          dot[u] = fmaf(qv.w, kv.w, dot[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kPerThread; ++u) {
        const int i = kg * kPerThread + u;
        float pv = 0.f;
        if (key_ok && i < nq) {
          const float b = bp + qc_bias(rt[time_bucket_i64(s_t[i] - tk, p.sub_bits, p.nb_t)]);
          pv = silu_exact(fmaf(p.alpha, dot[u], b));
          pv = b == kQcHidden ? 0.f : pv;
        }
        sp[kj * kPPitch + i] = pv;
      }
    } else {
#pragma unroll
      for (int u = 0; u < kPerThread; ++u) sp[kj * kPPitch + kg * kPerThread + u] = 0.f;
    }
    __syncthreads();
    if (p.weight_rows > 0 && tid < nk) {
      float w = 0.f;
#pragma unroll
      for (int i = 0; i < kQ; ++i) w += fabsf(sp[tid * kPPitch + i]);
      p.wpart[sq.wp0 + (int64_t(it.qtile) * H + h) * sq.len + jb + tid] = w;
    }
    const int quads = (nq + 3) >> 2;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int e = e0 + a * kThreads;
      if (e < dv) {
        for (int j = paired ? tid >> 6 : 0; j < nk; j += paired ? 2 : 1) {
          const float vv = sv[j * dv + e];
#pragma unroll
          for (int i = 0; i < kQ / 4; ++i) {
            if (i < quads) {
              const float4 pv = *reinterpret_cast<const float4 *>(sp + j * kPPitch + 4 * i);
              acc[a][4 * i] = fmaf(pv.x, vv, acc[a][4 * i]);
              acc[a][4 * i + 1] = fmaf(pv.y, vv, acc[a][4 * i + 1]);
              acc[a][4 * i + 2] = fmaf(pv.z, vv, acc[a][4 * i + 2]);
              acc[a][4 * i + 3] = fmaf(pv.w, vv, acc[a][4 * i + 3]);
            }
          }
        }
      }
    }
  }
  if (paired) {   // the odd keys' sums join the even ones'
    __syncthreads();
    if (tid >= 64 && e0 < dv)
#pragma unroll
      for (int i = 0; i < kQ; ++i) sv[i * 64 + e0] = acc[0][i];
    __syncthreads();
    if (tid < 64 && e0 < dv)
#pragma unroll
      for (int i = 0; i < kQ; ++i) acc[0][i] += sv[i * 64 + e0];
  }
  // ---- the candidate's own pair (distance 0 in position and time) ----
  __syncthreads();
  if (it.split == 0) {
    const T *k = static_cast<const T *>(p.k);
    const int warp = tid >> 5, lane = tid & 31;
    for (int i = warp; i < nq; i += kThreads / 32) {
      const T *kr = k + (sq.q0 + i0 + i) * p.k_rs + int64_t(h) * dq;
      float dot = 0.f;
      for (int e = lane; e < dq; e += 32) dot = fmaf(sq_q[i * dq + e], qc_float<T>(kr[e]), dot);
#pragma unroll
      for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
      const float b = qc_bias(rp[0]) + qc_bias(rt[0]);
      if (lane == 0) sp[i] = b == kQcHidden ? kQcNoOwn : silu_exact(fmaf(p.alpha, dot, b));
    }
  }
  __syncthreads();
  const T *v = static_cast<const T *>(p.v);
  T *out = static_cast<T *>(p.out);
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const int e = tid + a * kThreads;
    if (e >= dv) continue;   // (paired: the upper threads' e is past d_v)
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      if (i >= nq) break;
      const int64_t row = sq.q0 + i0 + i;
      float o = acc[a][i];
      if (it.split == 0 && sp[i] != kQcNoOwn)
        o = fmaf(sp[i], qc_float<T>(v[row * p.v_rs + int64_t(h) * dv + e]), o);
      if (sq.splits > 1)
        p.acc[(sq.acc0 + (int64_t(it.split) * sq.n + i0 + i) * H + h) * dv + e] = o;
      else if (p.out_f32)
        static_cast<float *>(p.out)[row * p.o_rs + int64_t(h) * dv + e] = o * p.scale;
      else
        out[row * p.o_rs + int64_t(h) * dv + e] = qc_round<T>(o * p.scale);
    }
  }
}

// ---------------------------------------------------------------------------
// Summing pass.  Blocks [0, out_blocks): one warp per (candidate, head) row of
// a split sequence adds its key ranges in order; the rest: one thread per
// cached row adds the weight partials over planes and heads in order.  The
// order is fixed, so results do not depend on which CTA finished first.  Bound by
// latency: 4 to 8 us.
// ---------------------------------------------------------------------------
constexpr int kFinThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kFinThreads)
    finish_kernel(const __grid_constant__ QcAttnParams p, int out_blocks, int plane) {
  const QCacheView &c = p.cache;
  const int H = c.heads, dv = c.d_v;
  if (int(blockIdx.x) < out_blocks) {
    const int row = int(blockIdx.x) * (kFinThreads / 32) + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= p.fin_rows) return;
    const int si = qc_find(p.seqs, p.n_seqs, row, [](const QcAttnSeq &s) { return s.fin0; });
    const QcAttnSeq &sq = p.seqs[si];
    const int x = row - sq.fin0;                       // i H + h
    const int64_t step = int64_t(sq.n) * H * dv;
    const float *a = p.acc + (sq.acc0 + x) * dv;
    T *o = static_cast<T *>(p.out) + (sq.q0 + x / H) * p.o_rs + int64_t(x % H) * dv;
    // four features per lane (d_v is a multiple of 32); eight key ranges' loads in flight
    for (int e = lane * 4; e < dv; e += 128) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      int k = 0;
      for (; k + 8 <= sq.splits; k += 8) {
        float4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
          v[u] = *reinterpret_cast<const float4 *>(a + (k + u) * step + e);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          s.x += v[u].x;
          s.y += v[u].y;
          s.z += v[u].z;
          s.w += v[u].w;
        }
      }
      for (; k < sq.splits; ++k) {
        const float4 v = *reinterpret_cast<const float4 *>(a + k * step + e);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      o[e] = qc_round<T>(s.x * p.scale);
      o[e + 1] = qc_round<T>(s.y * p.scale);
      o[e + 2] = qc_round<T>(s.z * p.scale);
      o[e + 3] = qc_round<T>(s.w * p.scale);
    }
    return;
  }
  const int64_t w = (int64_t(blockIdx.x) - out_blocks) * kFinThreads + threadIdx.x;
  if (w >= p.weight_rows) return;
  const int si = qc_find(p.seqs, p.n_seqs, w, [](const QcAttnSeq &s) { return s.wrow0; });
  const QcAttnSeq &sq = p.seqs[si];
  const int64_t j = w - sq.wrow0;
  const int planes = (sq.n + plane - 1) / plane * H;
  float s = 0.f;
  const float *wp = p.wpart + sq.wp0 + j;
#pragma unroll 8
  for (int k = 0; k < planes; ++k) s += wp[int64_t(k) * sq.len];
  float *dst = c.weight + sq.row + j;
  const float old = p.decay == 0.f ? 0.f : p.decay * *dst;
  *dst = fmaf(p.scale, s, old);
}

}  // namespace qc_simt

cudaError_t launch_qcache_attn_simt(const QcAttnParams &p, bool bf16, cudaStream_t st) {
  using namespace qc_simt;
  const size_t smem = smem_floats(p.cache.d_qk, p.cache.d_v) * sizeof(float);
  static PerDeviceOnce attr_b, attr_f;
  const size_t most = smem_floats(256, 256) * sizeof(float);
  cudaError_t e = bf16 ? set_smem_once(attr_b, attn_kernel<__nv_bfloat16>, most)
                       : set_smem_once(attr_f, attn_kernel<float>, most);
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(p.items) * unsigned(p.cache.heads);
  if (bf16)
    attn_kernel<__nv_bfloat16><<<grid, kThreads, smem, st>>>(p);
  else
    attn_kernel<float><<<grid, kThreads, smem, st>>>(p);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_qcache_finish(const QcAttnParams &p, bool bf16, int plane, cudaStream_t st) {
  using namespace qc_simt;
  const int64_t ob = (p.fin_rows + kFinThreads / 32 - 1) / (kFinThreads / 32);
  const int64_t wb = (p.weight_rows + kFinThreads - 1) / kFinThreads;
  if (ob + wb == 0) return cudaSuccess;
  if (bf16 && !p.out_f32)
    finish_kernel<__nv_bfloat16><<<unsigned(ob + wb), kFinThreads, 0, st>>>(p, int(ob), plane);
  else
    finish_kernel<float><<<unsigned(ob + wb), kFinThreads, 0, st>>>(p, int(ob), plane);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hstu
