// qcache_attn_sm100.cu -- candidates against the 4-bit history cache on the
// tensor cores (tcgen05, tensor memory), bf16, d_qk = d_v in {64, 128}.
//
//   out_i = c (sum_j SiLU(x_ij) v_j + SiLU(x_ii) v_i),
//   x_ij = alpha <q_i, k_j> + rab_pos[P_b - pos_j] + rab_time[tb(t_i - t_j)]
//   w_j  <- decay w_j + c sum_{i, h} |SiLU(x_ij)|
//
// One CTA = one (sequence, head, NQ candidates, range of 128-key tiles); both
// products are turned so that a thread owns a key, not a candidate:
//   S^T = K Q^T   [128 keys x NQ],   O^T += V^T P^T   [d x NQ]
// Why: everything a key brings along is then one value per thread.  All
// candidates of a call sit at one position and mostly share one time, so the
// position bias, and nearly always the time bias, is a constant of the thread,
// and its weight sum over the candidates stays in a register.  It also keeps
// the tile 128 keys high for a single candidate (NQ only pads the N side).
//
//   warps 12-19  read codes (16 bytes = one group per load, two tiles ahead),
//                decode them exactly to bf16 and write K and V tiles in the
//                128-byte swizzle.
//   warp 0       issues the MMAs: S^T of the next tile ahead of O^T of this one.
//   warps 4-11   read S^T (thread = key; each warpgroup half of the
//                candidates), make P = SiLU(x), write P^T (bf16) to shared
//                memory, add up the weights; at the end write O.
//   warps 1-3    the candidates' own pairs <q_i, k_i> meanwhile.
// Tensor memory: S^T in [0, NQ) and [NQ, 2 NQ) by turns, O^T in [2 NQ, 3 NQ).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "qcache_attn.cuh"
#include "tile_common.cuh"

namespace hstu {
namespace qc_tc {

constexpr int kTile = kQcKeyTile;
constexpr int kThreads = 640;
constexpr int kElemThreads = 256;     // warps 4-11
constexpr int kDecThreads = 256;      // warps 12-19
constexpr int kTblT = 385;            // float-exponent table of the time bias, sub_bits <= 4
constexpr uint32_t kBoxBytes = kTile * 128;   // 128 rows of 64 bf16

template <int D, int NQ>
struct Cfg {
  static constexpr int kTileBytes = kTile * D * 2;
  // The K tile is free again as soon as S^T is done, well before P is; one
  // buffer does where two would not fit.
  static constexpr int kK = D == 128 && NQ == 128 ? 1 : 2;
  static constexpr int kV = 2, kP = 2;
  static constexpr int kPBytes = NQ / 64 * int(kBoxBytes);
  static constexpr uint32_t kTmemCols = NQ == 128 ? 512 : 256;
};

template <int D, int NQ>
struct Smem {
  using C = Cfg<D, NQ>;
  alignas(1024) uint8_t q[NQ * D * 2];
  alignas(1024) uint8_t k[C::kK][C::kTileBytes];
  alignas(1024) uint8_t v[C::kV][C::kTileBytes];
  alignas(1024) uint8_t p[C::kP][C::kPBytes];   // behind v: see the D = 64 note at issue_o
  alignas(16) int64_t tq[NQ];     // candidates' times
  alignas(16) float tqd[NQ];      // and relative to the earliest of them
  float p_self[NQ];
  float tbl_t[kTblT];
  int64_t tq_min, tq_max;
  uint64_t k_full[C::kK], k_empty[C::kK], v_full[C::kV], v_empty[C::kV];
  uint64_t s_full[2], p_full[C::kP], p_empty[C::kP];
  uint64_t self_full, o_full, drain;
  uint32_t tmem_base;
  uint32_t abort;                 // a wait of this CTA ran out
};

// Bounded wait.  The CTA's own flag, not the error word of the workspace, tells
// its other roles to leave: the word may hold anything until this call's first
// CTA has cleared it.
__device__ __forceinline__ bool wait_cta(uint64_t *bar, uint32_t parity, uint32_t *abort,
                                         const WaitCtl &w) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile uint32_t *>(abort) != 0) return false;
    if (globaltimer_ns() - t0 > w.limit_ns) {
      *reinterpret_cast<volatile uint32_t *>(abort) = 1;
      record_error(w.err, kDevErrTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_cta_warp(uint64_t *bar, uint32_t parity, uint32_t *abort,
                                              const WaitCtl &w) {
  return __all_sync(0xffffffffu, wait_cta(bar, parity, abort, w));
}

__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// SiLU of the logit x.  With weights (which are returned in float32) the
// quotient form, good to a few 2^-22; else h (1 + tanh h), h = x / 2, half the
// special-function work, its error below P's rounding to bf16.
template <bool WEIGHTS>
__device__ __forceinline__ float silu_of(float x) {
  if constexpr (WEIGHTS) {
    return x * rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * x));
  } else {
    return fmaf(x, tanh_approx(x), x);   // x already halved
  }
}

// How a thread finds the time bias of its key against the candidates.
enum : int { kTimeOne = 0, kTimeFloat = 1, kTimeInt = 2 };

// 32 candidates of one key: P as bf16 pairs, and the sum of |P| over the first
// `live` of them.
template <int D, int NQ, bool WEIGHTS, int MODE>
__device__ __forceinline__ void chunk32(const uint32_t (&s)[32], uint32_t (&pk)[16],
                                        const Smem<D, NQ> &sm, int c0, float a, float c,
                                        float base, int64_t tk, const float *rt, float half,
                                        int sub_bits, int nb_t, int live, float &wsum) {
  const int sh = 23 - sub_bits;
  const int32_t r0 = fast_r0(sub_bits);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float pv[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float x = fmaf(a, __uint_as_float(s[e + u]), c);
      if constexpr (MODE == kTimeFloat) {
        const int32_t rr = __float_as_int(base + sm.tqd[c0 + e + u]) >> sh;
        x += sm.tbl_t[(rr > r0 ? rr : r0) - r0];
      } else if constexpr (MODE == kTimeInt) {
        x += half * qc_bias(rt[time_bucket_i64(sm.tq[c0 + e + u] - tk, sub_bits, nb_t)]);
      }
      pv[u] = silu_of<WEIGHTS>(x);
      if constexpr (WEIGHTS) {
        if (live >= 32 || e + u < live) wsum += fabsf(pv[u]);
      }
    }
    pk[e / 2] = pack_bf16x2(pv[0], pv[1]);
  }
}

template <int D, int NQ, bool WEIGHTS>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ QcAttnParams p) {
  using C = Cfg<D, NQ>;
  extern __shared__ uint8_t smem_raw[];
  Smem<D, NQ> &sm = *reinterpret_cast<Smem<D, NQ> *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const QCacheView &cv = p.cache;
  const int H = cv.heads;
  const int item = int(blockIdx.x) / H, h = int(blockIdx.x) - item * H;
  // The first CTA clears the error word.  A CTA records one only after a wait
  // of at least a microsecond, long after the first CTA has started.
  if (p.clear_err && blockIdx.x == 0 && tid < 4) p.wait.err[tid] = 0;
  const QcItem it = qc_item(p, item);
  const QcAttnSeq sq = p.seqs[it.seq];
  const int i0 = it.qtile * NQ, nq = min(NQ, sq.n - i0);
  const int64_t q_row = sq.q0 + i0;
  const int n_tiles = it.t1 - it.t0;
  const float *rp = p.rab_p + (p.rab_per_head ? int64_t(h) * p.nb_p : 0);
  const float *rt = p.rab_t + (p.rab_per_head ? int64_t(h) * p.nb_t : 0);
  const float half = WEIGHTS ? 1.0f : 0.5f;     // the tanh form works on x / 2
  constexpr uint32_t kQHalf = NQ * 128;         // bytes of one 64-column box of Q

  // ---- start-up: queries in the K-major 128-byte swizzle, tables, barriers ----
  {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + q_row * p.q_rs + h * D;
    constexpr int kUnits = NQ * (D / 8);
    for (int x = tid; x < kUnits; x += kThreads) {
      const int r = x / (D / 8), u = x % (D / 8);
      uint4 val = make_uint4(0, 0, 0, 0);
      if (r < nq) {
        const __nv_bfloat16 *src = q + r * p.q_rs + u * 8;
        if (p.vec) {
          val = *reinterpret_cast<const uint4 *>(src);
        } else {
          uint16_t e[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = reinterpret_cast<const uint16_t *>(src)[i];
          val = make_uint4(e[0] | uint32_t(e[1]) << 16, e[2] | uint32_t(e[3]) << 16,
                           e[4] | uint32_t(e[5]) << 16, e[6] | uint32_t(e[7]) << 16);
        }
      }
      *reinterpret_cast<uint4 *>(sm.q + (u >> 3) * kQHalf + r * 128 + (((u & 7) ^ (r & 7)) << 4)) =
          val;
    }
    if (p.sub_bits <= 4) {
      const int n = fast_table_size(p.sub_bits);
      for (int x = tid; x < n; x += kThreads)
        sm.tbl_t[x] = half * qc_bias(rt[fast_table_bucket(x, p.sub_bits, p.nb_t)]);
    }
  }
  if (warp == 1) {
    // candidates' times, their range, and their distances to the earliest;
    // a padding candidate takes the first one's
    int64_t lo = INT64_MAX, hi = INT64_MIN;
    for (int i = lane; i < NQ; i += 32) {
      const int64_t t = p.cand_ts[q_row + (i < nq ? i : 0)];
      sm.tq[i] = t;
      lo = t < lo ? t : lo;
      hi = t > hi ? t : hi;
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) {
      const int64_t a = __shfl_xor_sync(0xffffffffu, lo, m), b = __shfl_xor_sync(0xffffffffu, hi, m);
      lo = a < lo ? a : lo;
      hi = b > hi ? b : hi;
    }
    __syncwarp();
    for (int i = lane; i < NQ; i += 32) sm.tqd[i] = float(sm.tq[i] - lo);
    if (lane == 0) {
      sm.tq_min = lo;
      sm.tq_max = hi;
    }
  }
  if (tid == 0) {
    for (int i = 0; i < C::kK; ++i) {
      mbar_init(&sm.k_full[i], kDecThreads);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < C::kV; ++i) {
      mbar_init(&sm.v_full[i], kDecThreads);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], kElemThreads);
      mbar_init(&sm.p_empty[i], 1);
    }
    mbar_init(&sm.self_full, 96);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(&sm.tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  fence_proxy_async_smem();   // the queries, ahead of the MMAs that read them
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp == 0) {
    // ===================== MMA issuer =====================
    if (elect_one() && n_tiles > 0) {
      constexpr uint32_t idesc_s = idesc_bf16(kTile, NQ, false, false);
      constexpr uint32_t idesc_o = idesc_bf16(128, NQ, true, true);
      const uint64_t dq = sdesc_sw128(smem_u32(sm.q), 16, 1024);
      auto issue_s = [&](int n) {
        const uint64_t dk = sdesc_sw128(smem_u32(sm.k[n % C::kK]), 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss(tmem + (n & 1) * NQ, dk + (((kk / 4) * kBoxBytes + (kk % 4) * 32) >> 4),
                  dq + (((kk / 4) * kQHalf + (kk % 4) * 32) >> 4), idesc_s, kk > 0);
        umma_commit(&sm.s_full[n & 1]);
        umma_commit(&sm.k_empty[n % C::kK]);
      };
      // D = 64: the instruction is 128 rows high all the same; rows 64-127 read
      // whatever lies one box behind the V tile (the next V tile or P, inside
      // this struct) and fill tensor-memory lanes that nobody reads.
      auto issue_o = [&](int n) {
        const uint64_t dv = sdesc_sw128(smem_u32(sm.v[n % C::kV]), kBoxBytes, 1024);
        const uint64_t dp = sdesc_sw128(smem_u32(sm.p[n % C::kP]), kBoxBytes, 1024);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          umma_ss(tmem + 2 * NQ, dv + ((kk * 16 * 128) >> 4), dp + ((kk * 16 * 128) >> 4),
                  idesc_o, (n > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&sm.v_empty[n % C::kV]);
        umma_commit(&sm.p_empty[n % C::kP]);
      };
      bool ok = wait_cta(&sm.k_full[0], 0, &sm.abort, p.wait);
      tc_fence_after();
      if (ok) issue_s(0);
      for (int n = 0; n < n_tiles && ok; ++n) {
        if (n + 1 < n_tiles) {
          // its S^T columns are free: P of tile n - 1 was waited for below
          ok = wait_cta(&sm.k_full[(n + 1) % C::kK], ((n + 1) / C::kK) & 1, &sm.abort, p.wait);
          if (!ok) break;
          tc_fence_after();
          issue_s(n + 1);
        }
        ok = wait_cta(&sm.v_full[n % C::kV], (n / C::kV) & 1, &sm.abort, p.wait) &&
             wait_cta(&sm.p_full[n % C::kP], (n / C::kP) & 1, &sm.abort, p.wait);
        if (!ok) break;
        tc_fence_after();
        issue_o(n);
      }
      umma_commit(&sm.o_full);
      umma_commit(&sm.drain);
      drain_bar(&sm.drain, 0, p.wait.err, 4000000000ull);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ===================== the candidates' own pairs =====================
    if (it.split == 0) {
      const float bias = qc_bias(rp[0]) + qc_bias(rt[0]);
      for (int i = warp - 1; i < nq; i += 3) {
        const __nv_bfloat16 *qr =
            static_cast<const __nv_bfloat16 *>(p.q) + (q_row + i) * p.q_rs + h * D;
        const __nv_bfloat16 *kr =
            static_cast<const __nv_bfloat16 *>(p.k) + (q_row + i) * p.k_rs + h * D;
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e)
          dot = fmaf(__bfloat162float(qr[e * 32 + lane]), __bfloat162float(kr[e * 32 + lane]), dot);
#pragma unroll
        for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
        if (lane == 0) sm.p_self[i] = silu_of<true>(fmaf(p.alpha, dot, bias));
      }
    }
    mbar_arrive(&sm.self_full);
  } else if (warp < 12) {
    // ===================== elementwise =====================
    const int wg = (warp - 4) >> 2, quad = warp & 3;
    const int key = quad * 32 + lane;
    const uint32_t lanes = tmem + (uint32_t(quad * 32) << 16);
    const float a = half * p.alpha;
    const int64_t t_lo = sm.tq_min, t_hi = sm.tq_max;
    constexpr int kCols = NQ / 2;
    const int c_first = wg * kCols, c_end = min(c_first + kCols, nq);   // empty for small nq
    bool ok = true;
    for (int n = 0; n < n_tiles; ++n) {
      const int32_t j = (it.t0 + n) * kTile + key;
      const bool valid = j < sq.len;
      // what this key brings along: position bias, and its time bias when it
      // is the same for all candidates
      int mode = kTimeOne;
      float c = 0.f, base = 0.f, wsum = 0.f;
      int64_t tk = 0;
      if (c_first < c_end) {
        const int64_t row = sq.row + (valid ? j : 0);
        tk = cv.times[row];
        c = half * qc_bias(rp[pos_bucket(int64_t(sq.pos) - cv.pos[row], p.nb_p)]);
        const int32_t b_lo = time_bucket_i64(t_lo - tk, p.sub_bits, p.nb_t);
        const int32_t b_hi = t_hi == t_lo ? b_lo : time_bucket_i64(t_hi - tk, p.sub_bits, p.nb_t);
        if (__all_sync(0xffffffffu, b_lo == b_hi || !valid)) {
          c += half * qc_bias(rt[b_lo]);
        } else {
          const int64_t lim = int64_t(1) << 24;
          const bool near = t_hi - tk < lim && t_lo - tk > -lim;   // float differences are exact
          mode = __all_sync(0xffffffffu, p.sub_bits <= 4 && (near || !valid)) ? kTimeFloat
                                                                              : kTimeInt;
          base = float(t_lo - tk);
        }
      }
      ok = wait_cta_warp(&sm.s_full[n & 1], (n >> 1) & 1, &sm.abort, p.wait);
      if (ok && n >= C::kP)
        ok = wait_cta_warp(&sm.p_empty[n % C::kP], ((n / C::kP) - 1) & 1, &sm.abort, p.wait);
      if (!ok) break;
      tc_fence_after();
      uint8_t *pt = sm.p[n % C::kP] + key * 128;
#pragma unroll 1
      for (int c0 = c_first; c0 < c_end; c0 += 32) {
        uint32_t r[32], pk[16];
        tmem_ld32(lanes + (n & 1) * NQ + c0, r);
        tmem_wait_ld(r);
        const int live = c_end - c0;
        if (mode == kTimeOne)
          chunk32<D, NQ, WEIGHTS, kTimeOne>(r, pk, sm, c0, a, c, base, tk, rt, half, p.sub_bits,
                                            p.nb_t, live, wsum);
        else if (mode == kTimeFloat)
          chunk32<D, NQ, WEIGHTS, kTimeFloat>(r, pk, sm, c0, a, c, base, tk, rt, half, p.sub_bits,
                                              p.nb_t, live, wsum);
        else
          chunk32<D, NQ, WEIGHTS, kTimeInt>(r, pk, sm, c0, a, c, base, tk, rt, half, p.sub_bits,
                                            p.nb_t, live, wsum);
        if (!valid) {
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0;
        }
        uint8_t *box = pt + (c0 >> 6) * kBoxBytes;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<uint4 *>(box + (((((c0 & 63) >> 3) + e) ^ (key & 7)) << 4)) =
              make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
      }
      tc_fence_before();          // S^T has been read
      fence_proxy_async_smem();   // P^T is written
      mbar_arrive(&sm.p_full[n % C::kP]);
      if constexpr (WEIGHTS) {
        if (valid && c_first < c_end)
          p.wpart[sq.wp0 + (int64_t(it.qtile * 2 + wg) * H + h) * sq.len + j] = wsum;
      }
    }
    // ---- O^T (tensor memory: lane = feature) + own pair -> rows of out ----
    if (ok) ok = wait_cta_warp(&sm.self_full, 0, &sm.abort, p.wait);
    if (ok && n_tiles > 0) ok = wait_cta_warp(&sm.o_full, 0, &sm.abort, p.wait);
    tc_fence_after();
    if (ok && key < D) {
      const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v) + q_row * p.v_rs + h * D + key;
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + q_row * p.o_rs + h * D + key;
      float *acc = p.acc + ((sq.acc0 + (int64_t(it.split) * sq.n + i0) * H + h) * D + key);
#pragma unroll 1
      for (int c0 = c_first; c0 < c_end; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(lanes + 2 * NQ + c0, r);
        tmem_wait_ld(r);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int i = c0 + e;
          if (i < c_end) {
            float o = n_tiles > 0 ? __uint_as_float(r[e]) : 0.f;
            if (it.split == 0) o = fmaf(sm.p_self[i], __bfloat162float(v[i * p.v_rs]), o);
            if (sq.splits > 1)
              acc[int64_t(i) * H * D] = o;
            else
              out[i * p.o_rs] = __float2bfloat16_rn(o * p.scale);
          }
        }
      }
    }
  } else {
    // ===================== decoding K and V =====================
    constexpr int G = D / 32, kPer = kTile * G / kDecThreads;   // groups per row / per thread
    const int dt = tid - 384;
    const uint4 *kc = reinterpret_cast<const uint4 *>(cv.k_codes);
    const uint4 *vc = reinterpret_cast<const uint4 *>(cv.v_codes);
    const int64_t g0 = (int64_t(h) * cv.rows + sq.row) * G;
    struct Raw {
      uint4 k[kPer], v[kPer];
      uint32_t kp[kPer], vp[kPer];
    };
    // rows behind the sequence's last decode to zeros: scale 0
    auto fetch = [&](int n, Raw &r) {
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        const int idx = dt + x * kDecThreads;
        const int64_t j = int64_t(it.t0 + n) * kTile + idx / G;
        r.k[x] = r.v[x] = make_uint4(0, 0, 0, 0);
        r.kp[x] = r.vp[x] = 0;
        if (n < n_tiles && j < sq.len) {
          const int64_t at = g0 + int64_t(it.t0 + n) * kTile * G + idx;
          r.k[x] = ld_stream(kc + at);
          r.v[x] = ld_stream(vc + at);
          r.kp[x] = cv.k_scales[at];
          r.vp[x] = cv.v_scales[at];
        }
      }
    };
    auto store = [&](uint8_t *tile, const uint4 (&code)[kPer], const uint32_t (&par)[kPer]) {
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        const int idx = dt + x * kDecThreads, row = idx / G, g = idx % G;
        uint32_t zz, ss;
        q4_group(par[x], zz, ss);
        // A warp's eight 16-byte stores of a phase hold 2 rows x 4 groups at
        // D = 128; groups 2 and 3 (the other box, same banks) go in another
        // chunk order so that the phase touches every bank once.
        const bool swap = G == 4 && (g & 2);
        const uint32_t w[4] = {swap ? code[x].z : code[x].x, swap ? code[x].w : code[x].y,
                               swap ? code[x].x : code[x].z, swap ? code[x].y : code[x].w};
        uint8_t *dst = tile + (g >> 1) * kBoxBytes + row * 128;
        const int first = (g & 1) * 4, flip = swap ? 2 : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t o[4];
          q4_decode_bf16(w[e], zz, ss, o);
          *reinterpret_cast<uint4 *>(dst + (((first + (e ^ flip)) ^ (row & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    };
    Raw raw[2];
    fetch(0, raw[0]);
    fetch(1, raw[1]);
    bool ok = true;
    auto step = [&](int n, Raw &r) {
      if (n >= C::kK)
        ok = wait_cta_warp(&sm.k_empty[n % C::kK], ((n / C::kK) - 1) & 1, &sm.abort, p.wait);
      if (!ok) return;
      store(sm.k[n % C::kK], r.k, r.kp);
      fence_proxy_async_smem();
      mbar_arrive(&sm.k_full[n % C::kK]);
      if (n >= C::kV)
        ok = wait_cta_warp(&sm.v_empty[n % C::kV], ((n / C::kV) - 1) & 1, &sm.abort, p.wait);
      if (!ok) return;
      store(sm.v[n % C::kV], r.v, r.vp);
      fence_proxy_async_smem();
      mbar_arrive(&sm.v_full[n % C::kV]);
      fetch(n + 2, r);
    };
    for (int n = 0; n < n_tiles && ok; n += 2) {
      step(n, raw[0]);
      if (ok && n + 1 < n_tiles) step(n + 1, raw[1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int D, int NQ, bool WEIGHTS>
cudaError_t launch_t(const QcAttnParams &p, cudaStream_t st) {
  constexpr size_t smem = sizeof(Smem<D, NQ>) + 1024;
  static_assert(smem <= 232448, "shared memory");
  static PerDeviceOnce attr;
  cudaError_t e = set_smem_once(attr, attn_kernel<D, NQ, WEIGHTS>, smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(p.items) * unsigned(p.cache.heads);
  attn_kernel<D, NQ, WEIGHTS><<<grid, kThreads, smem, st>>>(p);
  count_launch();
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const QcAttnParams &p, int nq, cudaStream_t st) {
  const bool w = p.weight_rows > 0;
  if (nq == 64) return w ? launch_t<D, 64, true>(p, st) : launch_t<D, 64, false>(p, st);
  return w ? launch_t<D, 128, true>(p, st) : launch_t<D, 128, false>(p, st);
}

}  // namespace qc_tc

cudaError_t launch_qcache_attn_tc(const QcAttnParams &p, int nq, cudaStream_t st) {
  return p.cache.d_qk == 64 ? qc_tc::launch_d<64>(p, nq, st) : qc_tc::launch_d<128>(p, nq, st);
}

}  // namespace hstu
