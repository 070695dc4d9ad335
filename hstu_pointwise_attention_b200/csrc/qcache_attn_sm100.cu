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
//   warps 4-11   two warpgroups, taking tiles by turns: read S^T (thread = key),
//                make P = SiLU(x), write P^T (bf16) to shared memory, add up the
//                weights.  Before that the candidates' own pairs <q_i, k_i>, at
//                the end each warpgroup writes half of O.
//   warps 1-3    a tile per warp, up to four tiles ahead: what each key brings
//                along (KeyBias).
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

// How the time bias of a tile's keys is found.  kTimeOne: the same for all
// candidates, part of c.  kTimeTwo: each key meets one or two neighbouring
// buckets, c below and c2 from candidate time t on (relative to the earliest).
// kTimeFloat: by the float-exponent table, t = earliest candidate - key.
// kTimeInt: bucket by bucket in 64 bits.
enum : int { kTimeOne = 0, kTimeTwo = 1, kTimeFloat = 2, kTimeInt = 3 };
constexpr int kBias = 4;              // tiles of KeyBias in flight
struct KeyBias {
  float c[kTile], c2[kTile], t[kTile];
  int64_t tk[kTile];
  int mode;
};

template <int D, int NQ>
struct Smem {
  using C = Cfg<D, NQ>;
  alignas(1024) uint8_t q[NQ * D * 2];
  alignas(1024) uint8_t k[C::kK][C::kTileBytes];
  alignas(1024) uint8_t v[C::kV][C::kTileBytes];
  alignas(1024) uint8_t p[C::kP][C::kPBytes];   // behind v: see the D = 64 note at issue_o
  KeyBias bias[kBias];
  alignas(16) int64_t tq[NQ];     // candidates' times
  alignas(16) float tqd[NQ];      // and relative to the earliest of them
  float p_self[NQ];
  float tbl_t[kTblT];
  int64_t tq_min, tq_max;
  uint64_t k_full[C::kK], k_empty[C::kK], v_full[C::kV], v_empty[C::kV];
  uint64_t s_full[2], p_full[C::kP], p_empty[C::kP];
  uint64_t bias_full[kBias], bias_empty[kBias];
  uint64_t o_full, drain;
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
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
// 8 values of a bf16 row.
__device__ __forceinline__ uint4 load_row8(const __nv_bfloat16 *src, bool vec) {
  if (vec) return *reinterpret_cast<const uint4 *>(src);
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = reinterpret_cast<const uint16_t *>(src)[i];
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}
__device__ __forceinline__ float dot8(const uint4 &a, const uint4 &b, float s) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
    s = fmaf(__uint_as_float(x[i] & 0xFFFF0000u), __uint_as_float(y[i] & 0xFFFF0000u), s);
  }
  return s;
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

// W candidates of one key: P = SiLU(x) as bf16 pairs and, with weights, the sum
// of |P| over the first `live` of them.  With weights (returned in float32)
// SiLU is x / (1 + 2^y), y = -x log2 e, good to a few 2^-22; else h (1 + tanh h)
// with h = x / 2, half the special-function work, its error below P's rounding.
template <int D, int NQ, bool WEIGHTS, int MODE, bool ALL, int W>
__device__ __forceinline__ void chunk(const uint32_t (&s)[W], uint32_t (&pk)[W / 2],
                                        const Smem<D, NQ> &sm, int c0, float a, float c, float c2,
                                        float t, int64_t tk, const float *rt, float half,
                                        int sub_bits, int nb_t, int live, float &wsum) {
  const int sh = 23 - sub_bits;
  const int32_t r0 = fast_r0(sub_bits);
  constexpr float kL = -1.4426950408889634f;
  const float ay = kL * a, cy = kL * c;
  float tq[4];
#pragma unroll
  for (int e = 0; e < W; e += 2) {
    if constexpr (MODE == kTimeTwo || MODE == kTimeFloat) {
      if ((e & 3) == 0) {
        const float4 v = *reinterpret_cast<const float4 *>(&sm.tqd[c0 + e]);
        tq[0] = v.x;
        tq[1] = v.y;
        tq[2] = v.z;
        tq[3] = v.w;
      }
    }
    float pv[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float sv = __uint_as_float(s[e + u]);
      float x, y = 0.f;
      if constexpr (MODE == kTimeOne) {
        x = fmaf(a, sv, c);
        if constexpr (WEIGHTS) y = fmaf(ay, sv, cy);
      } else if constexpr (MODE == kTimeTwo) {
        x = fmaf(a, sv, tq[(e & 3) + u] >= t ? c2 : c);
        y = kL * x;
      } else if constexpr (MODE == kTimeFloat) {
        const int32_t rr = __float_as_int(t + tq[(e & 3) + u]) >> sh;
        x = fmaf(a, sv, c) + sm.tbl_t[(rr > r0 ? rr : r0) - r0];
        y = kL * x;
      } else {
        x = fmaf(a, sv, c) +
            half * qc_bias(rt[time_bucket_i64(sm.tq[c0 + e + u] - tk, sub_bits, nb_t)]);
        y = kL * x;
      }
      if constexpr (WEIGHTS) {
        pv[u] = x * rcp_approx(1.0f + ex2_approx(y));
        if (ALL || e + u < live) wsum += fabsf(pv[u]);
      } else {
        pv[u] = fmaf(x, tanh_approx(x), x);   // x already halved
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
      if (r < nq) val = load_row8(q + r * p.q_rs + u * 8, p.vec);
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
      mbar_init(&sm.p_full[i], kElemThreads / 2);
      mbar_init(&sm.p_empty[i], 1);
    }
    for (int i = 0; i < kBias; ++i) {
      mbar_init(&sm.bias_full[i], 32);
      mbar_init(&sm.bias_empty[i], kElemThreads / 64);
    }
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
    // ===================== what each key brings along =====================
    const int64_t t_lo = sm.tq_min, t_hi = sm.tq_max, lim = int64_t(1) << 24;
    const int sh = 23 - p.sub_bits;
    const int32_t r0 = fast_r0(p.sub_bits);
    for (int n = warp - 1; n < n_tiles; n += 3) {
      KeyBias &kb = sm.bias[n % kBias];
      int64_t tk[4];
      float c[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        // keys behind the last take its values; their P is zeroed
        const int32_t j = min((it.t0 + n) * kTile + x * 32 + lane, sq.len - 1);
        tk[x] = cv.times[sq.row + j];
        c[x] = __int_as_float(cv.pos[sq.row + j]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x)
        c[x] = half * qc_bias(rp[pos_bucket(int64_t(sq.pos) - __float_as_int(c[x]), p.nb_p)]);
      // float time differences are exact: every one, and its two parts, below 2^24
      bool one = true, near = p.sub_bits <= 4 && t_hi - t_lo < lim;
      int32_t b_lo[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        b_lo[x] = time_bucket_i64(t_lo - tk[x], p.sub_bits, p.nb_t);
        if (t_hi != t_lo)
          one = one && b_lo[x] == time_bucket_i64(t_hi - tk[x], p.sub_bits, p.nb_t);
        near = near && t_hi - tk[x] < lim && t_lo - tk[x] > -lim;
      }
      one = __all_sync(0xffffffffu, one);
      near = __all_sync(0xffffffffu, near);
      if (n >= kBias &&
          !wait_cta_warp(&sm.bias_empty[n % kBias], ((n / kBias) - 1) & 1, &sm.abort, p.wait))
        break;
      int mode = one ? kTimeOne : near ? kTimeFloat : kTimeInt;
      if (one) {
#pragma unroll
        for (int x = 0; x < 4; ++x) c[x] += half * qc_bias(rt[b_lo[x]]);
      } else if (near) {
        // table entries of the earliest and the latest candidate
        float base[4];
        int32_t e_lo[4], e_hi[4];
        bool two = true;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          base[x] = float(t_lo - tk[x]);
          e_lo[x] = max(__float_as_int(base[x]) >> sh, r0) - r0;
          e_hi[x] = max(__float_as_int(float(t_hi - tk[x])) >> sh, r0) - r0;
          two = two && e_hi[x] - e_lo[x] <= 1;
        }
        if (__all_sync(0xffffffffu, two)) {
          // The entry is e_lo + 1 exactly from the distance on whose bits are
          // (e_lo + 1 + r0) << sh: an integer below 2^24 where both entries
          // occur, so its difference to base is exact.
          mode = kTimeTwo;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            kb.c2[x * 32 + lane] = c[x] + sm.tbl_t[e_hi[x]];
            kb.t[x * 32 + lane] = __int_as_float((e_lo[x] + 1 + r0) << sh) - base[x];
            c[x] += sm.tbl_t[e_lo[x]];
          }
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) kb.t[x * 32 + lane] = base[x];
        }
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        kb.c[x * 32 + lane] = c[x];
        kb.tk[x * 32 + lane] = tk[x];
      }
      if (lane == 0) kb.mode = mode;
      mbar_arrive(&sm.bias_full[n % kBias]);
    }
  } else if (warp < 12) {
    // ===================== elementwise =====================
    const int wg = (warp - 4) >> 2, quad = warp & 3;
    const int key = quad * 32 + lane;
    const uint32_t lanes = tmem + (uint32_t(quad * 32) << 16);
    if (it.split == 0) {
      // The candidates' own pairs, while the first tiles are decoded: 8 lanes
      // per candidate, each NQ / 8 of them per warp; every load is issued ahead
      // of the first sum.
      constexpr int kPass = NQ / 32, kVec = D / 64;
      const int sub = lane & 7;
      uint4 qv[kPass][kVec], kv[kPass][kVec];
#pragma unroll
      for (int x = 0; x < kPass; ++x) {
        const int i = (warp - 4) * (NQ / 8) + x * 4 + (lane >> 3);
#pragma unroll
        for (int y = 0; y < kVec; ++y) {
          qv[x][y] = kv[x][y] = make_uint4(0, 0, 0, 0);
          if (i < nq) {
            const int64_t e = h * D + (y * 8 + sub) * 8;
            qv[x][y] = load_row8(static_cast<const __nv_bfloat16 *>(p.q) + (q_row + i) * p.q_rs + e,
                                 p.vec);
            kv[x][y] = load_row8(static_cast<const __nv_bfloat16 *>(p.k) + (q_row + i) * p.k_rs + e,
                                 p.vec);
          }
        }
      }
      const float bias = qc_bias(rp[0]) + qc_bias(rt[0]);
#pragma unroll
      for (int x = 0; x < kPass; ++x) {
        float dot = 0.f;
#pragma unroll
        for (int y = 0; y < kVec; ++y) dot = dot8(qv[x][y], kv[x][y], dot);
#pragma unroll
        for (int m = 4; m; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
        const float xs = fmaf(p.alpha, dot, bias);
        if (sub == 0)
          sm.p_self[(warp - 4) * (NQ / 8) + x * 4 + (lane >> 3)] =
              xs * rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * xs));
      }
    }
    const float a = half * p.alpha;
    bool ok = true;
    for (int n = wg; n < n_tiles; n += 2) {
      const int32_t j = (it.t0 + n) * kTile + key;
      const bool valid = j < sq.len;
      const KeyBias &kb = sm.bias[n % kBias];
      ok = wait_cta_warp(&sm.bias_full[n % kBias], (n / kBias) & 1, &sm.abort, p.wait);
      if (!ok) break;
      const int mode = kb.mode;
      const float c = kb.c[key];
      float c2 = 0.f, t = 0.f, wsum = 0.f;
      int64_t tk = 0;
      if (mode != kTimeOne) {
        c2 = kb.c2[key];
        t = kb.t[key];
        tk = kb.tk[key];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.bias_empty[n % kBias]);
      ok = wait_cta_warp(&sm.s_full[wg], (n >> 1) & 1, &sm.abort, p.wait);
      if (ok && n >= C::kP)   // the product of the tile two back has read P
        ok = wait_cta_warp(&sm.p_empty[wg], ((n >> 1) - 1) & 1, &sm.abort, p.wait);
      if (!ok) break;
      tc_fence_after();
      uint8_t *pt = sm.p[wg] + key * 128;
#define HSTU_QC_CHUNK(M_, A_, W_)                                                                \
  chunk<D, NQ, WEIGHTS, M_, A_, W_>(r, pk, sm, c0, a, c, c2, t, tk, rt, half, p.sub_bits, p.nb_t, \
                                    nq - c0, wsum)
      if (nq <= 16 && mode == kTimeOne) {   // few candidates: half a chunk
        constexpr int c0 = 0;
        uint32_t r[16], pk[8];
        tmem_ld16(lanes + wg * NQ, r);
        tmem_wait_ld(r);
        HSTU_QC_CHUNK(kTimeOne, !WEIGHTS, 16);
#pragma unroll
        for (int e = 0; e < 8; ++e) pk[e] = valid ? pk[e] : 0;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<uint4 *>(pt + ((e ^ (key & 7)) << 4)) =
              make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
      } else {
#pragma unroll 1
        for (int c0 = 0; c0 < nq; c0 += 32) {
          uint32_t r[32], pk[16];
          tmem_ld32(lanes + wg * NQ + c0, r);
          tmem_wait_ld(r);
          if (mode == kTimeOne) {
            if (!WEIGHTS || nq - c0 >= 32)
              HSTU_QC_CHUNK(kTimeOne, true, 32);
            else
              HSTU_QC_CHUNK(kTimeOne, false, 32);
          } else if (mode == kTimeTwo) {
            HSTU_QC_CHUNK(kTimeTwo, !WEIGHTS, 32);
          } else if (mode == kTimeFloat) {
            HSTU_QC_CHUNK(kTimeFloat, !WEIGHTS, 32);
          } else {
            HSTU_QC_CHUNK(kTimeInt, !WEIGHTS, 32);
          }
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
      }
#undef HSTU_QC_CHUNK
      tc_fence_before();          // S^T has been read
      fence_proxy_async_smem();   // P^T is written
      mbar_arrive(&sm.p_full[wg]);
      if constexpr (WEIGHTS) {
        if (valid) p.wpart[sq.wp0 + (int64_t(it.qtile) * H + h) * sq.len + j] = wsum;
      }
    }
    // ---- O^T (tensor memory: lane = feature) + own pair -> rows of out ----
    named_bar_sync(1, kElemThreads);   // p_self of all warps
    constexpr int kCols = NQ / 2;
    const int c_first = wg * kCols, c_end = min(c_first + kCols, nq);
    if (ok && n_tiles > 0) ok = wait_cta_warp(&sm.o_full, 0, &sm.abort, p.wait);
    tc_fence_after();
    if (ok && quad * 32 < D) {
      const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.v) + q_row * p.v_rs + h * D + key;
      __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out) + q_row * p.o_rs + h * D + key;
      float *acc = p.acc + ((sq.acc0 + (int64_t(it.split) * sq.n + i0) * H + h) * D + key);
#pragma unroll 1
      for (int c0 = c_first; c0 < c_end; c0 += 16) {
        uint32_t r[16];
        tmem_ld16(lanes + 2 * NQ + c0, r);
        tmem_wait_ld(r);
        float o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          o[e] = n_tiles > 0 ? __uint_as_float(r[e]) : 0.f;
          if (it.split == 0 && c0 + e < c_end)
            o[e] = fmaf(sm.p_self[c0 + e], __bfloat162float(v[(c0 + e) * p.v_rs]), o[e]);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int i = c0 + e;
          if (i < c_end) {
            if (sq.splits > 1)
              acc[int64_t(i) * H * D] = o[e];
            else
              out[i * p.o_rs] = __float2bfloat16_rn(o[e] * p.scale);
          }
        }
      }
    }
  } else {
    // ===================== decoding K and V =====================
    // A warp takes 8 rows x 4 groups (16 x 2 at D = 64) of a tile, 512 bytes in
    // one piece.  Eight lanes that store together hold 4 rows x 2 neighbouring
    // groups, whose 16-byte chunks lie in eight different banks under the
    // swizzle.
    constexpr int G = D / 32;                      // groups per row
    constexpr int kPer = kTile * G / kDecThreads;  // groups per thread and tile
    constexpr int kStep = kDecThreads / G;         // rows between a thread's groups
    const int dw = warp - 12;
    const int row = G == 4 ? dw * 8 + ((lane >> 4) << 2) + ((lane >> 1) & 3)
                           : dw * 16 + (lane >> 1);
    const int g = G == 4 ? ((lane >> 3) & 1) * 2 + (lane & 1) : lane & 1;
    const int64_t at = (int64_t(h) * cv.rows + sq.row + int64_t(it.t0) * kTile + row) * G + g;
    const uint4 *kc = reinterpret_cast<const uint4 *>(cv.k_codes) + at;
    const uint4 *vc = reinterpret_cast<const uint4 *>(cv.v_codes) + at;
    const uint16_t *ks = cv.k_scales + at, *vs = cv.v_scales + at;
    int32_t left = sq.len - it.t0 * kTile - row;   // rows of the sequence from this one on
    uint32_t off[4];   // where the group's chunks go in a tile
#pragma unroll
    for (int e = 0; e < 4; ++e)
      off[e] = (g >> 1) * kBoxBytes + row * 128 + ((((g & 1) * 4 + e) ^ (row & 7)) << 4);
    struct Raw {
      uint4 k[kPer], v[kPer];
      uint32_t kp[kPer], vp[kPer];
    };
    auto fetch = [&](Raw &r) {
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        if (x * kStep < left) {
          r.k[x] = ld_stream(kc + x * kDecThreads);
          r.v[x] = ld_stream(vc + x * kDecThreads);
          r.kp[x] = ks[x * kDecThreads];
          r.vp[x] = vs[x * kDecThreads];
        } else {   // behind the last row: zeros
          r.k[x] = r.v[x] = make_uint4(0, 0, 0, 0);
          r.kp[x] = r.vp[x] = 0;
        }
      }
      kc += kTile * G;
      vc += kTile * G;
      ks += kTile * G;
      vs += kTile * G;
      left -= kTile;
    };
    auto store = [&](uint32_t tile, const uint4 (&code)[kPer], const uint32_t (&par)[kPer]) {
#pragma unroll
      for (int x = 0; x < kPer; ++x) {
        uint32_t zz, ss;
        q4_group(par[x], zz, ss);
        const uint32_t w[4] = {code[x].x, code[x].y, code[x].z, code[x].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t o[4];
          q4_decode_bf16(w[e], zz, ss, o);
          st_shared_v4(tile + off[e] + x * kStep * 128, o);
        }
      }
    };
    const uint32_t k0 = smem_u32(sm.k[0]), v0 = smem_u32(sm.v[0]);
    Raw raw[2];
    fetch(raw[0]);
    fetch(raw[1]);
    bool ok = true;
    auto step = [&](int n, Raw &r) {
      if (n >= C::kK)
        ok = wait_cta_warp(&sm.k_empty[n % C::kK], ((n / C::kK) - 1) & 1, &sm.abort, p.wait);
      if (!ok) return;
      store(k0 + (n % C::kK) * C::kTileBytes, r.k, r.kp);
      fence_proxy_async_smem();
      mbar_arrive(&sm.k_full[n % C::kK]);
      if (n >= C::kV)
        ok = wait_cta_warp(&sm.v_empty[n % C::kV], ((n / C::kV) - 1) & 1, &sm.abort, p.wait);
      if (!ok) return;
      store(v0 + (n % C::kV) * C::kTileBytes, r.v, r.vp);
      fence_proxy_async_smem();
      mbar_arrive(&sm.v_full[n % C::kV]);
      fetch(r);
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
