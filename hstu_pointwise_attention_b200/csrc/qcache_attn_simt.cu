// qcache_attn_simt.cu -- candidates against the 4-bit history cache on the
// CUDA cores (any head size, float32 or bf16), and the summing pass of both
// attention kernels.
//
//   out_i = c (sum_j SiLU(x_ij) v_j + SiLU(x_ii) v_i),
//   x_ij = alpha <q_i, k_j> + rab_pos[P_b - pos_j] + rab_time[tb(t_i - t_j)]
//   w_j  <- decay w_j + c sum_{i, h} |SiLU(x_ij)|
//
// One CTA = 16 candidates of one (sequence, head) and a range of keys, 32 keys
// at a time: rows of the cache are decoded to float32 in shared memory, each
// thread makes the weights of one key for 4 candidates, then each thread sums
// one or two output columns over the 32 keys.  It is bound by its shared-memory
// reads (one per multiply-add in the first step).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qcache_attn.cuh"

namespace hstu {
namespace qc_simt {

constexpr int kThreads = 128;
constexpr int kQ = kQcSimtQueries;   // candidates per CTA
constexpr int kKeys = 32;            // keys per step
constexpr int kPerThread = kQ / (kThreads / kKeys);

// Shared memory in floats: q [kQ][d_qk], k [kKeys][d_qk + 1], v [kKeys][d_v],
// p [kQ][kKeys + 1].
__host__ __device__ constexpr size_t smem_floats(int d_qk, int d_v) {
  return size_t(kQ) * d_qk + size_t(kKeys) * (d_qk + 1) + size_t(kKeys) * d_v + kQ * (kKeys + 1);
}

__device__ __forceinline__ float silu_exact(float x) { return x / (1.0f + expf(-x)); }

template <typename T>
__global__ void __launch_bounds__(kThreads)
    attn_kernel(const __grid_constant__ QcAttnParams p) {
  extern __shared__ float sm[];
  const QCacheView &c = p.cache;
  const int H = c.heads, dq = c.d_qk, dv = c.d_v;
  const int item = int(blockIdx.x) / H, h = int(blockIdx.x) - item * H;
  const int tid = threadIdx.x;
  if (p.clear_err && blockIdx.x == 0 && tid < 4) p.wait.err[tid] = 0;
  const QcItem it = qc_item(p, item);
  const QcAttnSeq &sq = p.seqs[it.seq];
  const int i0 = it.qtile * kQ, nq = min(kQ, sq.n - i0);
  float *sq_q = sm, *sk = sq_q + kQ * dq, *sv = sk + kKeys * (dq + 1), *sp = sv + kKeys * dv;
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
  const int32_t j_end = min(it.t1 * kQcKeyTile, sq.len);
  for (int32_t jb = it.t0 * kQcKeyTile; jb < j_end; jb += kKeys) {
    const int nk = min(kKeys, j_end - jb);
    __syncthreads();
    // decode 32 keys and values: a word of 8 codes per thread and step
    const int64_t at0 = int64_t(h) * c.rows + sq.row + jb;
    for (int x = tid; x < kKeys * (dq >> 3); x += kThreads) {
      const int r = x / (dq >> 3), w = x - r * (dq >> 3);
      uint32_t code = 0, par = 0;
      if (r < nk) {
        code = c.k_codes[(at0 + r) * (dq >> 3) + w];
        par = c.k_scales[(at0 + r) * (dq >> 5) + (w >> 2)];
      }
      const float s = q4_scale(par);
      const int z = int(par & 15u);
#pragma unroll
      for (int e = 0; e < 8; ++e) sk[r * (dq + 1) + 8 * w + e] = s * float(q4_code(code, e) - z);
    }
    for (int x = tid; x < kKeys * (dv >> 3); x += kThreads) {
      const int r = x / (dv >> 3), w = x - r * (dv >> 3);
      uint32_t code = 0, par = 0;
      if (r < nk) {
        code = c.v_codes[(at0 + r) * (dv >> 3) + w];
        par = c.v_scales[(at0 + r) * (dv >> 5) + (w >> 2)];
      }
      const float s = q4_scale(par);
      const int z = int(par & 15u);
#pragma unroll
      for (int e = 0; e < 8; ++e) sv[r * dv + 8 * w + e] = s * float(q4_code(code, e) - z);
    }
    __syncthreads();
    {
      float dot[kPerThread];
#pragma unroll
      for (int u = 0; u < kPerThread; ++u) dot[u] = 0.f;
      const float *kr = sk + kj * (dq + 1), *qr = sq_q + kg * kPerThread * dq;
      for (int e = 0; e < dq; ++e) {
        const float kv = kr[e];
#pragma unroll
        for (int u = 0; u < kPerThread; ++u) dot[u] = fmaf(qr[u * dq + e], kv, dot[u]);
      }
      const bool key_ok = kj < nk;
      const int64_t row = sq.row + jb + (key_ok ? kj : 0);
      const float bp = rp[pos_bucket(int64_t(sq.pos) - c.pos[row], p.nb_p)];
      const int64_t tk = c.times[row];
#pragma unroll
      for (int u = 0; u < kPerThread; ++u) {
        const int i = kg * kPerThread + u;
        const float b = qc_bias(bp + rt[time_bucket_i64(s_t[i] - tk, p.sub_bits, p.nb_t)]);
        const float x = fmaf(p.alpha, dot[u], b);
        sp[i * (kKeys + 1) + kj] = key_ok && i < nq ? silu_exact(x) : 0.f;
      }
    }
    __syncthreads();
    if (p.weight_rows > 0 && tid < nk) {
      float w = 0.f;
#pragma unroll
      for (int i = 0; i < kQ; ++i) w += fabsf(sp[i * (kKeys + 1) + tid]);
      p.wpart[sq.wp0 + (int64_t(it.qtile) * H + h) * sq.len + jb + tid] = w;
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const int e = tid + a * kThreads;
      if (e < dv) {
        for (int j = 0; j < nk; ++j) {
          const float vv = sv[j * dv + e];
#pragma unroll
          for (int i = 0; i < kQ; ++i) acc[a][i] = fmaf(sp[i * (kKeys + 1) + j], vv, acc[a][i]);
        }
      }
    }
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
      if (lane == 0) sp[i] = silu_exact(fmaf(p.alpha, dot, qc_bias(rp[0] + rt[0])));
    }
  }
  __syncthreads();
  const T *v = static_cast<const T *>(p.v);
  T *out = static_cast<T *>(p.out);
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const int e = tid + a * kThreads;
    if (e >= dv) continue;
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
      if (i >= nq) break;
      const int64_t row = sq.q0 + i0 + i;
      float o = acc[a][i];
      if (it.split == 0) o = fmaf(sp[i], qc_float<T>(v[row * p.v_rs + int64_t(h) * dv + e]), o);
      if (sq.splits > 1)
        p.acc[(sq.acc0 + (int64_t(it.split) * sq.n + i0 + i) * H + h) * dv + e] = o;
      else
        out[row * p.o_rs + int64_t(h) * dv + e] = qc_round<T>(o * p.scale);
    }
  }
}

// ---------------------------------------------------------------------------
// Summing pass.  Blocks [0, out_blocks): one warp per (candidate, head) row of
// a split sequence adds its key ranges in order; the rest: one thread per
// cached row adds the weight partials over planes and heads in order.  The
// order is fixed, so results do not depend on which CTA finished first.
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
  if (bf16)
    finish_kernel<__nv_bfloat16><<<unsigned(ob + wb), kFinThreads, 0, st>>>(p, int(ob), plane);
  else
    finish_kernel<float><<<unsigned(ob + wb), kFinThreads, 0, st>>>(p, int(ob), plane);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hstu
