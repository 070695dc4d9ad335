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
//   warp 0       issues the MMAs as their operands arrive.
//   warps 1-3    a tile per warp, up to six tiles ahead: what each key brings
//                along (KeyBias).
//   then 8 or 16 elementwise warps: one or two warpgroups take a tile, the next
//                ones the next: read S^T (thread = key, 64 candidates), make
//                P = SiLU(x), write P^T (bf16) to shared memory, add up the
//                weights; at the end each warpgroup writes 32 candidates of O.
//   then 8 or 4 warps for keys: bring codes to shared memory (cp.async, ahead),
//                decode them exactly to bf16 and write K to tensor memory
//                (lane = key), from where the MMA takes it;
//   and as many for values the same way, V to shared memory in the 128-byte
//                swizzle.
// The candidates' own pairs stay out of the products: the sum over keys of a
// tile adds 0 v_i to every other candidate, so an infinity in one candidate's v
// would reach all of them.  The elementwise warps make SiLU(x_ii) while they wait
// for the first S^T, and SiLU(x_ii) v_i joins O where it is written.
// K stays out of shared memory, whose traffic would bound the loop (an
// MMA with both operands there and N = 128 takes all of its 128 bytes a cycle):
// that saves 32 KB written and 32 KB read of about 260 KB per tile at D = 128,
// NQ = 128.
// Tensor memory: S^T slots, then O^T, then two K tiles (Cfg).
//
// Bound by the elementwise warps and their hand-overs: at 128 candidates each of the
// two groups works on its tile of 128 x 128 pairs and then waits for the next S^T
// (tensor memory has room for two, so one is made while the other is read; a slot is
// free once its last columns are in registers: with the wait for P in its place 8 x 256
// took 3 us longer and 4 x 1,024 6).  Measured (8 heads of 128): 8 histories of 4,096
// with 256 candidates and weights 72 us and 7 more to sum (477 TFLOP/s; issue slots
// 77 %, special functions 50 %, tensor cores 25 % busy); 4 of 8,192 with 1,024 candidates
// 234 us (588 TFLOP/s; 74 %, 33 %, 32 %).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "qcache_attn.cuh"
#include "tile_common.cuh"

namespace hstu {
namespace qc_tc {

constexpr int kTile = kQcKeyTile;
constexpr int kThreads = 896;         // 4 control, 24 elementwise and decoding warps
constexpr int kTblT = 385;            // float-exponent table of the time bias, sub_bits <= 4
constexpr uint32_t kBoxBytes = kTile * 128;   // 128 rows of 64 bf16

template <int D, int NQ>
struct Cfg {
  // With up to 64 candidates the decoding is most of the work, with up to 128 the
  // elementwise pass: 64 candidates of a tile per elementwise warpgroup, two tiles
  // in work, and the other warps decode, half of them K, half V.
  static constexpr int kHalves = NQ / 64;                   // warpgroups per tile
  static constexpr int kElemWarps = 8 * kHalves;
  static constexpr int kDecWarps = (24 - kElemWarps) / 2;   // per operand: 8 or 4
  static constexpr int kDecThreads = 32 * kDecWarps;
  static constexpr int kG = D / 32;                         // groups per row
  static constexpr int kPer = kTile * kG / kDecThreads;     // groups per thread and tile
  static constexpr int kParBytes = kPer == 1 ? 4 : 2 * kPer;   // K: parameters copied per thread
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kV = 2;
  // Tiles of P: with two a warpgroup waited for the product of its last tile (4 x
  // 1,024 candidates 240 us, with three 233).
  static constexpr int kP = 3;
  static constexpr int kPBytes = NQ / 64 * int(kBoxBytes);
  // Tiles of codes on their way: with few candidates the cache's bandwidth is
  // the limit, and bytes in flight per SM = bandwidth x latency, about 36 KB at
  // full HBM rate; with many a tile's time covers the latency.
  static constexpr int kStages = D == 128 ? (NQ == 128 ? 1 : 3) : 4;
  static constexpr int kCodeBytes = kTile * D / 2;       // of one tile of K (or V)
  static constexpr int kScaleBytes = kTile * 8;          // 8 bytes per row (V at D = 64: 4 of them)
  // Tensor memory columns: kS slots of S^T, O^T, two K tiles.
  static constexpr int kS = NQ == 128 ? 2 : 3;
  static constexpr uint32_t kO = kS * NQ, kK = kO + NQ;
  static_assert(kK + 2 * (D / 2) <= 512, "tensor memory");
};

// How the time bias of 32 keys of a tile is found.  kTimeOne: the same for all
// candidates, part of c.  kTimeTwo: each key meets one or two neighbouring
// buckets, both hidden or neither, c below and c2 from candidate time t on
// (relative to the earliest).
// kTimeFloat: by the float-exponent table, t = earliest candidate - key.
// kTimeInt: bucket by bucket in 64 bits.
enum : int { kTimeOne = 0, kTimeTwo = 1, kTimeFloat = 2, kTimeInt = 3 };
// Tiles of KeyBias in flight: a multiple of the 3 warps that fill them and of
// the 2 warpgroups that take them, so a slot always has the same two parties and
// none of them can be a whole round of its barriers ahead of the other (a parity
// wait cannot tell two rounds apart).
constexpr int kBias = 6;
struct KeyBias {
  float c[kTile], c2[kTile], t[kTile];
  int mode[4];   // of 32 keys each
};

template <int D, int NQ>
struct Smem {
  using C = Cfg<D, NQ>;
  alignas(1024) uint8_t q[NQ * D * 2];
  alignas(1024) uint8_t v[C::kV][C::kTileBytes];
  alignas(1024) uint8_t p[C::kP][C::kPBytes];       // behind v: see the D = 64 note at issue_o
  alignas(16) uint8_t k_codes[C::kStages][C::kCodeBytes];
  alignas(16) uint8_t v_codes[C::kStages][C::kCodeBytes];
  alignas(16) uint8_t k_scales[C::kStages][C::kScaleBytes];
  alignas(16) uint8_t v_scales[C::kStages][C::kScaleBytes];
  KeyBias bias[kBias];
  alignas(16) float tqd[NQ];      // candidates' times relative to the earliest of them
  float own[NQ];                  // SiLU of the candidates' own pairs (first key range only)
  float tbl_t[kTblT];
  int64_t tq_min, tq_max;
  uint64_t k_full[2], k_empty[2], v_full[C::kV], v_empty[C::kV];
  uint64_t s_full[3];             // with three slots a warpgroup takes every other round of one:
                                  // the commits are in order, so the round between is over by then
  uint64_t s_empty[3];            // the warpgroup has read S^T
  uint64_t p_full[C::kP], p_empty[C::kP];
  uint64_t bias_full[kBias], bias_empty[kBias];
  uint64_t q_full, o_full, drain;
  uint32_t tmem_base;
  uint32_t abort;                 // a wait of this CTA ran out
  static_assert(sizeof(p) >= NQ * D * sizeof(float), "O goes through the P tiles at the end");
};

// Bounded wait.  The CTA's own flag, not the error word of the workspace, tells
// its other roles to leave: the word may hold anything until this call's first
// CTA has cleared it.
// The roles' loops run side by side on every scheduler and together have to stay
// in the instruction cache: what a loop seldom needs (here, finding a segment) is
// kept out of line.
__device__ __noinline__ bool wait_cta_slow(uint64_t *bar, uint32_t parity, uint32_t *abort,
                                           uint32_t *err, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile uint32_t *>(abort) != 0) return false;
    if (globaltimer_ns() - t0 > limit_ns) {
      *reinterpret_cast<volatile uint32_t *>(abort) = 1;
      record_error(err, kDevErrTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_cta(uint64_t *bar, uint32_t parity, uint32_t *abort,
                                         const WaitCtl &w) {
  return mbar_try_wait(bar, parity) || wait_cta_slow(bar, parity, abort, w.err, w.limit_ns);
}
__device__ __forceinline__ bool wait_cta_warp(uint64_t *bar, uint32_t parity, uint32_t *abort,
                                              const WaitCtl &w) {
  return __all_sync(0xffffffffu, wait_cta(bar, parity, abort, w));
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint32_t *v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
// The time bias of one pair, bucket by bucket (times too far apart for floats).
__device__ __noinline__ float time_bias_int(int64_t dt, const float *rt, int sub_bits, int nb_t) {
  return qc_bias(rt[time_bucket_i64(dt, sub_bits, nb_t)]);
}

// acc plus the products of two bf16 pairs.
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float acc) {
  acc = fmaf(__uint_as_float(a << 16), __uint_as_float(b << 16), acc);
  return fmaf(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u), acc);
}

// SiLU of a halved logit: by tanh, far below zero by the quotient.
__device__ __forceinline__ float silu_tanh(float h) { return fmaf(h, tanh_approx(h), h); }
__device__ __forceinline__ float silu_half(float h) {
  return h < -3.5f ? qc_silu(h + h) : silu_tanh(h);
}
// Of four (out of line: seldom needed).
__device__ __noinline__ float4 silu_half4(float a, float b, float c, float d) {
  return make_float4(silu_half(a), silu_half(b), silu_half(c), silu_half(d));
}

// 16 candidates of one key: P = SiLU(x) as bf16 pairs and, with weights, the sum of
// |P|, ahead of its rounding, over the candidates.
//   With weights SiLU is its quotient (qc_silu).  A reciprocal for every pair: two pairs
//   that share one are NaN together, and sharing saves no time (8 x 256 candidates 82.1 us
//   shared, 81.3 not).
//   Without, it is h (1 + tanh h), h = x / 2, half the special-function work (4 x 1,024
//   candidates 219 us, by the quotient 263).  Its sum cancels for negative x: at 2^20
//   points of every unit of [-20, 12) the approximate tanh left SiLU at most 1e-5 off,
//   from -7 up at most 0.035 of P's rounding to bf16, but below -8 up to 2.2 of it and at
//   -16 all of P.  So logits below -7 go by the quotient (looking for them costs 7 us).
template <int D, int NQ, bool WEIGHTS, int MODE>
__device__ __forceinline__ void chunk(const uint32_t (&s)[16], uint32_t (&pk)[8],
                                      const Smem<D, NQ> &sm, int c0, float a, float c,
                                      float c2, float t, int64_t tk, const float *rt, float half,
                                      int sub_bits, int nb_t, const int64_t *ts, int nq,
                                      float &wsum) {
  const int sh = 23 - sub_bits;
  const int32_t r0 = fast_r0(sub_bits);
  float x[16], pv[16];
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    float4 tq = make_float4(0.f, 0.f, 0.f, 0.f);
    if constexpr (MODE == kTimeTwo || MODE == kTimeFloat)
      tq = *reinterpret_cast<const float4 *>(&sm.tqd[c0 + e]);
    const float tqs[4] = {tq.x, tq.y, tq.z, tq.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float sv = __uint_as_float(s[e + u]);
      if constexpr (MODE == kTimeOne) {
        x[e + u] = fmaf(a, sv, c);
      } else if constexpr (MODE == kTimeTwo) {
        x[e + u] = fmaf(a, sv, tqs[u] >= t ? c2 : c);
      } else if constexpr (MODE == kTimeFloat) {
        const int32_t rr = __float_as_int(t + tqs[u]) >> sh;
        const float b = c + sm.tbl_t[(rr > r0 ? rr : r0) - r0];
        x[e + u] = b == kQcHidden ? 0.f : fmaf(a, sv, b);   // SiLU(0) = 0
      } else {
        const float b = c + half * time_bias_int(ts[min(c0 + e + u, nq - 1)] - tk, rt, sub_bits,
                                                 nb_t);
        x[e + u] = b == kQcHidden ? 0.f : fmaf(a, sv, b);
      }
    }
  }
  if constexpr (WEIGHTS) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      pv[e] = qc_silu(x[e]);
      // padding has the bias of its key: left out, since 0 times it could be NaN
      if (c0 + e < nq) wsum += fabsf(pv[e]);
    }
  } else {   // x halved
    float lo = x[0];
#pragma unroll
    for (int e = 1; e < 15; e += 2) lo = fminf(fminf(lo, x[e]), x[e + 1]);
    lo = fminf(lo, x[15]);
#pragma unroll
    for (int e = 0; e < 16; ++e) pv[e] = silu_tanh(x[e]);
    if (lo < -3.5f) {
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 y = silu_half4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        pv[e] = y.x;
        pv[e + 1] = y.y;
        pv[e + 2] = y.z;
        pv[e + 3] = y.w;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 16; e += 2) pk[e / 2] = pack_bf16x2(pv[e], pv[e + 1]);
}

// The decoding warps of K (IS_V false) or V: tiles of codes from the cache into
// stages (cp.async), from there to bf16, K to tensor memory, V to shared memory.
//   K: thread = key and half of the row (or all of it), since a warp writes its own 32 lanes of
//   tensor memory; a row's chunks are permuted in the stage so that 8 lanes that
//   read together touch every bank once.
//   V: a warp takes 8 rows x 4 groups (16 x 2 at D = 64), 512 bytes in one piece;
//   eight lanes that store together hold 4 rows x 2 neighbouring groups, whose
//   16-byte chunks lie in eight different banks under the swizzle.
template <int D, int NQ, bool IS_V>
__device__ __forceinline__ void decode_tiles(const QcAttnParams &p, Smem<D, NQ> &sm,
                                             const QcItem &it, const QcAttnSeq &sq, int h,
                                             uint32_t tmem, int dw, int lane) {
  using C = Cfg<D, NQ>;
  constexpr int G = C::kG, kPer = C::kPer, kDecThreads = C::kDecThreads;
  constexpr int kStep = kDecThreads / G;         // V: rows between a thread's groups
  const QCacheView &cv = p.cache;
  const int dt = dw * 32 + lane, hx = dw >> 2;
  const int n_tiles = it.t1 - it.t0;
  const int row = !IS_V    ? (dw & 3) * 32 + lane
                  : G == 4 ? dw * 8 + ((lane >> 4) << 2) + ((lane >> 1) & 3)
                           : dw * 16 + (lane >> 1);
  const int g = !IS_V ? hx * kPer : G == 4 ? ((lane >> 3) & 1) * 2 + (lane & 1) : lane & 1;
  const int64_t at = (int64_t(h) * cv.rows + sq.row + int64_t(it.t0) * kTile + row) * G + g;
  const uint8_t *const src0 = reinterpret_cast<const uint8_t *>(IS_V ? cv.v_codes : cv.k_codes);
  const uint8_t *const psrc0 = reinterpret_cast<const uint8_t *>(IS_V ? cv.v_scales : cv.k_scales);
  const uint8_t *src = src0 + at * 16;
  // parameters travel 4 bytes and more at a time: K the thread's groups (a single
  // one with its neighbour), V a whole row through the lane of its first group
  const uint8_t *psrc = psrc0 + (at - (!IS_V && kPer == 1 ? (g & 1) : 0)) * 2;
  int32_t left = sq.len - it.t0 * kTile - row;   // the sequence's rows from this one on
  uint8_t *const codes = IS_V ? sm.v_codes[0] : sm.k_codes[0];
  uint8_t *const scales = IS_V ? sm.v_scales[0] : sm.k_scales[0];
  uint32_t code_at[kPer];   // where the thread's codes lie in a stage
#pragma unroll
  for (int x = 0; x < kPer; ++x)
    code_at[x] = IS_V     ? (x * kDecThreads + dt) * 16
                 : G == 4 ? row * 64 + (((g + x) ^ ((row >> 1) & 3)) << 4)
                          : row * 32 + (((g + x) ^ ((row >> 2) & 1)) << 4);
  const uint32_t scale_at = IS_V ? row * 2 * G : (hx * kTile + row) * C::kParBytes;
  const uint32_t code_dst = smem_u32(codes), scale_dst = smem_u32(scales) + scale_at;
  auto copy = [&](int st) {   // the next tile of the cache into stage st
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const bool ok = (IS_V ? x * kStep : 0) < left;
      cp_async<16>(code_dst + st * C::kCodeBytes + code_at[x],
                   ok ? src + (IS_V ? x * kDecThreads : x) * 16 : src0, ok);
      if (IS_V && g == 0)
        cp_async<2 * G>(scale_dst + st * C::kScaleBytes + x * kStep * 2 * G,
                        ok ? psrc + x * kDecThreads * 2 : psrc0, ok);
    }
    if (!IS_V)
      cp_async<C::kParBytes>(scale_dst + st * C::kScaleBytes, 0 < left ? psrc : psrc0, 0 < left);
    src += kTile * G * 16;
    psrc += kTile * G * 2;
    left -= kTile;
  };
  int m_copy = 0;
#pragma unroll 1
  for (; m_copy < C::kStages; ++m_copy) {
    if (m_copy < n_tiles) copy(m_copy);
    cp_async_commit();
  }
  uint64_t *const full = IS_V ? sm.v_full : sm.k_full;
  uint64_t *const empty = IS_V ? sm.v_empty : sm.k_empty;
  uint32_t off[4];   // V: where the group's chunks go in a tile
#pragma unroll
  for (int e = 0; e < 4; ++e)
    off[e] = smem_u32(sm.v[0]) + (g >> 1) * kBoxBytes + row * 128 +
             ((((g & 1) * 4 + e) ^ (row & 7)) << 4);
  const uint32_t k_tile = tmem + (uint32_t((dw & 3) * 32) << 16) + C::kK + hx * (kPer * 16);
  // 32 values of group x to their place in tile buffer `buf`
  auto put = [&](int buf, int x, const uint32_t (&o)[16]) {
    if constexpr (IS_V) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        st_shared_v4(off[e] + buf * C::kTileBytes + x * kStep * 128, &o[4 * e]);
    } else {
      tmem_st16(k_tile + buf * (D / 2) + x * 16, o);
    }
  };
  auto done = [&](int buf) {
    if constexpr (IS_V) {
      fence_proxy_async_smem();
    } else {
      tmem_wait_st();
      tc_fence_before();
    }
    mbar_arrive(&full[buf]);
  };
  int st = 0;
#pragma unroll 1
  for (int n = 0; n < n_tiles; ++n) {
    const int buf = n & 1;
    cp_async_wait<C::kStages - 1>();
    if (IS_V) __syncwarp();   // the row's parameters came through another lane of this warp
    uint4 code[kPer];
    uint32_t par[kPer];
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      code[x] = *reinterpret_cast<const uint4 *>(codes + st * C::kCodeBytes + code_at[x]);
      par[x] = *reinterpret_cast<const uint16_t *>(
          scales + st * C::kScaleBytes + scale_at +
          (IS_V ? x * kStep * 2 * G + g * 2 : kPer == 1 ? (g & 1) * 2 : x * 2));
    }
    __syncwarp();   // the warp has read the stage
    if (m_copy < n_tiles) copy(st);
    cp_async_commit();
    ++m_copy;
    st = st == C::kStages - 1 ? 0 : st + 1;
    if (n >= 2 &&
        !wait_cta_warp(&empty[buf], ((n >> 1) - 1) & 1, &sm.abort, p.wait))
      break;
    if (!IS_V) tc_fence_after();
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      uint32_t zz, ss, o[16];
      q4_group(par[x], zz, ss);
      const uint32_t w[4] = {code[x].x, code[x].y, code[x].z, code[x].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t v4[4];
        q4_decode_bf16(w[e], zz, ss, v4);
#pragma unroll
        for (int u = 0; u < 4; ++u) o[4 * e + u] = v4[u];
      }
      put(buf, x, o);
    }
    done(buf);
  }
  cp_async_wait<0>();
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

  if (tid == 64) {
    mbar_init(&sm.q_full, 32 * C::kElemWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], C::kDecThreads);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], C::kDecThreads);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_empty[i], 128 * C::kHalves);
    }
    for (int i = 0; i < C::kP; ++i) {
      mbar_init(&sm.p_full[i], 128 * C::kHalves);
      mbar_init(&sm.p_empty[i], 1);
    }
    for (int i = 0; i < kBias; ++i) {
      mbar_init(&sm.bias_full[i], 32);
      mbar_init(&sm.bias_empty[i], 4 * C::kHalves);
    }
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp < 4) {
    if (warp == 0) {
      // ===================== MMA issuer =====================
      if (elect_one()) {
        constexpr uint32_t idesc_s = idesc_bf16(kTile, NQ, false, false);
        constexpr uint32_t idesc_o = idesc_bf16(128, NQ, true, true);
        const uint64_t dq = sdesc_sw128(smem_u32(sm.q), 16, 1024);
        bool ok = wait_cta(&sm.q_full, 0, &sm.abort, p.wait);
        int ns = 0, no = 0;               // next S^T, next O^T
        int s_slot = 0, s_par = 0;        // ns % kS, (ns / kS) & 1
        int p_slot = 0, p_par = 0;        // no % kP, (no / kP) & 1
        uint32_t idle = 0;
        uint64_t t0 = 0;
        while (ok && no < n_tiles) {
          // S^T first: the warpgroup that takes it may be waiting
          if (ns < n_tiles && mbar_test_wait(&sm.k_full[ns & 1], (ns >> 1) & 1) &&
              (ns < C::kS || mbar_test_wait(&sm.s_empty[s_slot], s_par ^ 1))) {
            tc_fence_after();
            const uint32_t k = tmem + C::kK + (ns & 1) * (D / 2);
#pragma unroll 2
            for (int kk = 0; kk < D / 16; ++kk)
              umma_ts(tmem + s_slot * NQ, k + kk * 8, dq + (((kk / 4) * kQHalf + (kk % 4) * 32) >> 4),
                      idesc_s, kk > 0);
            umma_commit(&sm.s_full[s_slot]);
            umma_commit(&sm.k_empty[ns & 1]);
            if (++s_slot == C::kS) {
              s_slot = 0;
              s_par ^= 1;
            }
            ++ns;
            idle = 0;
          } else if (no < ns && mbar_test_wait(&sm.p_full[p_slot], p_par) &&
                     mbar_test_wait(&sm.v_full[no & 1], (no >> 1) & 1)) {
            // D = 64: the instruction is 128 rows high all the same; rows 64-127
            // read whatever lies one box behind the V tile (the next V tile or P,
            // inside this struct) and fill tensor-memory lanes that nobody reads.
            tc_fence_after();
            const uint64_t dv = sdesc_sw128(smem_u32(sm.v[no & 1]), kBoxBytes, 1024);
            const uint64_t dp = sdesc_sw128(smem_u32(sm.p[p_slot]), kBoxBytes, 1024);
#pragma unroll 2
            for (int kk = 0; kk < kTile / 16; ++kk)
              umma_ss(tmem + C::kO, dv + ((kk * 16 * 128) >> 4), dp + ((kk * 16 * 128) >> 4),
                      idesc_o, (no > 0 || kk > 0) ? 1u : 0u);
            umma_commit(&sm.v_empty[no & 1]);
            umma_commit(&sm.p_empty[p_slot]);
            if (++p_slot == C::kP) {
              p_slot = 0;
              p_par ^= 1;
            }
            ++no;
            idle = 0;
          } else if ((++idle & 63) == 0) {   // bounded, like wait_cta
            if (idle == 64) t0 = globaltimer_ns();
            if (*reinterpret_cast<volatile uint32_t *>(&sm.abort) != 0) ok = false;
            if (ok && globaltimer_ns() - t0 > p.wait.limit_ns) {
              *reinterpret_cast<volatile uint32_t *>(&sm.abort) = 1;
              record_error(p.wait.err, kDevErrTimeout);
              ok = false;
            }
          }
        }
        umma_commit(&sm.o_full);
        umma_commit(&sm.drain);
        drain_bar(&sm.drain, 0, p.wait.err, 4000000000ull);
      }
      __syncwarp();
    } else {
      // ===================== what each key brings along =====================
      if (warp == 1) {
        // candidates' times, their range, and their distances to the earliest;
        // a padding candidate takes the first one's
        int64_t lo = INT64_MAX, hi = INT64_MIN, t[NQ / 32];
#pragma unroll
        for (int i = 0; i < NQ / 32; ++i) {
          t[i] = p.cand_ts[q_row + (i * 32 + lane < nq ? i * 32 + lane : 0)];
          lo = t[i] < lo ? t[i] : lo;
          hi = t[i] > hi ? t[i] : hi;
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) {
          const int64_t a = __shfl_xor_sync(0xffffffffu, lo, m);
          const int64_t b = __shfl_xor_sync(0xffffffffu, hi, m);
          lo = a < lo ? a : lo;
          hi = b > hi ? b : hi;
        }
#pragma unroll
        for (int i = 0; i < NQ / 32; ++i) {
          sm.tqd[i * 32 + lane] = float(t[i] - lo);
        }
        if (lane == 0) {
          sm.tq_min = lo;
          sm.tq_max = hi;
        }
      }
      named_bar_sync(2, 96);
      const int64_t t_lo = sm.tq_min, t_hi = sm.tq_max, lim = int64_t(1) << 24;
      const int sh = 23 - p.sub_bits;
      const int32_t r0 = fast_r0(p.sub_bits);
      if (t_lo != t_hi && p.sub_bits <= 4) {   // candidates of several times: the exponent table
        const int n = fast_table_size(p.sub_bits);
        for (int x = tid - 32; x < n; x += 96)
          sm.tbl_t[x] = half * qc_bias(rt[fast_table_bucket(x, p.sub_bits, p.nb_t)]);
        named_bar_sync(2, 96);
      }
#pragma unroll 1
      for (int n = warp - 1; n < n_tiles; n += 3) {
        KeyBias &kb = sm.bias[n % kBias];
        if (n >= kBias &&
            !wait_cta_warp(&sm.bias_empty[n % kBias], ((n / kBias) - 1) & 1, &sm.abort, p.wait))
          break;
        // 32 keys (one quadrant) at a time, the next ones' rows on their way;
        // keys behind the last take its values (their P is zeroed)
        auto row_of = [&](int x) {
          return sq.row + min((it.t0 + n) * kTile + x * 32 + lane, sq.len - 1);
        };
        int64_t tk = cv.times[row_of(0)];
        int32_t pk = cv.pos[row_of(0)];
#pragma unroll 1
        for (int x = 0; x < 4; ++x) {
          const int64_t t = tk;
          float c = half * qc_bias(rp[pos_bucket(int64_t(sq.pos) - pk, p.nb_p)]);
          if (x < 3) {
            tk = cv.times[row_of(x + 1)];
            pk = cv.pos[row_of(x + 1)];
          }
          const int32_t b_lo = time_bucket_i64(t_lo - t, p.sub_bits, p.nb_t);
          int mode = kTimeOne;
          if (t_hi != t_lo &&
              !__all_sync(0xffffffffu, b_lo == time_bucket_i64(t_hi - t, p.sub_bits, p.nb_t))) {
            // float time differences are exact: every one, and its two parts, below 2^24
            const bool near = __all_sync(0xffffffffu, p.sub_bits <= 4 && t_hi - t_lo < lim &&
                                                          t_hi - t < lim && t_lo - t > -lim);
            mode = near ? kTimeFloat : kTimeInt;
          }
          if (mode == kTimeOne) {
            c += half * qc_bias(rt[b_lo]);
          } else if (mode == kTimeFloat) {
            // table entries of the earliest and the latest candidate
            const float base = float(t_lo - t);
            const int32_t e_lo = max(__float_as_int(base) >> sh, r0) - r0;
            const int32_t e_hi = max(__float_as_int(float(t_hi - t)) >> sh, r0) - r0;
            kb.t[x * 32 + lane] = base;
            const float c_lo = c + sm.tbl_t[e_lo], c_hi = c + sm.tbl_t[e_hi];
            if (__all_sync(0xffffffffu, e_hi - e_lo <= 1 &&
                                            (c_lo == kQcHidden) == (c_hi == kQcHidden))) {
              // The entry is e_lo + 1 exactly from the distance on whose bits are
              // (e_lo + 1 + r0) << sh: an integer below 2^24 where both entries
              // occur, so its difference to base is exact.
              mode = kTimeTwo;
              kb.c2[x * 32 + lane] = c_hi;
              kb.t[x * 32 + lane] = __int_as_float((e_lo + 1 + r0) << sh) - base;
              c = c_lo;
            }
          }
          kb.c[x * 32 + lane] = c;
          if (lane == 0) kb.mode[x] = mode;
        }
        mbar_arrive(&sm.bias_full[n % kBias]);
      }
    }
  } else if (warp < 4 + C::kElemWarps) {
    // ===================== elementwise =====================
    // warpgroup w takes tiles of parity `par` and candidates [64 hf, 64 hf + 64)
    const int w = (warp - 4) >> 2, par = w / C::kHalves, hf = w % C::kHalves, quad = warp & 3;
    const int key = quad * 32 + lane;
    const uint32_t lanes = tmem + (uint32_t(quad * 32) << 16);
    // The warpgroup's 32 candidates of Q and of the output: a thread takes chunk u (8
    // features) of rows r0 + x kRows.
    constexpr int kRowLanes = D / 8, kRows = 128 / kRowLanes;
    const int wt = (tid - 128) & 127, u = wt % kRowLanes, r0 = w * 32 + wt / kRowLanes;
    {
      // the queries, K-major in the 128-byte swizzle; rows behind the last are zero
      const __nv_bfloat16 *q =
          static_cast<const __nv_bfloat16 *>(p.q) + q_row * p.q_rs + h * D + u * 8;
#pragma unroll
      for (int x = 0; x < 32 / kRows; ++x) {
        const int r = r0 + x * kRows;
        uint4 val = make_uint4(0, 0, 0, 0);
        if (r < nq) val = load_row8(q + r * p.q_rs, p.vec);
        *reinterpret_cast<uint4 *>(sm.q + (u >> 3) * kQHalf + r * 128 +
                                   (((u & 7) ^ (r & 7)) << 4)) = val;
      }
      fence_proxy_async_smem();
      mbar_arrive(&sm.q_full);
    }
    // the candidates' own pairs (distance 0 in position and time)
    if (it.split == 0) {
      const __nv_bfloat16 *k =
          static_cast<const __nv_bfloat16 *>(p.k) + q_row * p.k_rs + h * D + u * 8;
      const float b0 = qc_bias(rp[0]) + qc_bias(rt[0]);
      // (unrolled at 128 candidates, its registers spill: 4 x 1,024 candidates 237 us, so 229)
#pragma unroll (NQ == 64 ? 4 : 1)
      for (int x = 0; x < 32 / kRows; ++x) {
        const int r = r0 + x * kRows;
        uint4 kw = make_uint4(0, 0, 0, 0);
        if (r < nq) kw = load_row8(k + r * p.k_rs, p.vec);
        const uint4 qw = *reinterpret_cast<const uint4 *>(
            sm.q + (u >> 3) * kQHalf + r * 128 + (((u & 7) ^ (r & 7)) << 4));
        float dot = dot2(qw.x, kw.x, 0.f);
        dot = dot2(qw.y, kw.y, dot);
        dot = dot2(qw.z, kw.z, dot);
        dot = dot2(qw.w, kw.w, dot);
#pragma unroll
        for (int m = 1; m < kRowLanes; m <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
        const float xs = fmaf(p.alpha, dot, b0);
        if (u == 0) sm.own[r] = b0 == kQcHidden ? kQcNoOwn : qc_silu(xs);
      }
    }
    const float a = half * p.alpha;
    bool ok = true;
    int slot = par, round = 0;           // n % kS, n / kS
    int p_slot = par, p_round = 0;       // n % kP, n / kP
#pragma unroll 1
    for (int n = par; n < n_tiles;
         n += 2, slot += 2, slot -= slot >= C::kS ? (++round, C::kS) : 0, p_slot += 2,
             p_slot -= p_slot >= C::kP ? (++p_round, C::kP) : 0) {
      const uint32_t s_col = lanes + slot * NQ;
      uint8_t *pt = sm.p[p_slot] + hf * kBoxBytes + key * 128;
      const int32_t j = (it.t0 + n) * kTile + key;
      const int bs = n % kBias;
      const KeyBias &kb = sm.bias[bs];
      ok = wait_cta_warp(&sm.bias_full[bs], (n / kBias) & 1, &sm.abort, p.wait);
      if (!ok) break;
      const int mode = kb.mode[quad];
      const float c = kb.c[key];
      // a key behind the last adds nothing, nor one whose buckets are hidden for all
      const bool valid = j < sq.len && c != kQcHidden;
      float c2 = 0.f, t = 0.f, wsum = 0.f;
      int64_t tk = 0;
      if (mode != kTimeOne) {
        c2 = kb.c2[key];
        t = kb.t[key];
        if (mode == kTimeInt) tk = cv.times[sq.row + min(j, sq.len - 1)];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.bias_empty[bs]);
      ok = wait_cta_warp(&sm.s_full[slot], round & 1, &sm.abort, p.wait);
      if (ok && n >= C::kP)   // the product of the tile kP back has read P
        ok = wait_cta_warp(&sm.p_empty[p_slot], (p_round - 1) & 1, &sm.abort, p.wait);
      if (!ok) break;
      tc_fence_after();
#define HSTU_QC_CHUNK(M_)                                                                       \
  chunk<D, NQ, WEIGHTS, M_>(r, pk, sm, c0, a, c, c2, t, tk, rt, half, p.sub_bits, p.nb_t, \
                        p.cand_ts + q_row, nq, wsum)
      const int c_end = min(hf * 64 + 64, nq);
      if (c_end <= hf * 64) mbar_arrive(&sm.s_empty[slot]);   // no candidate in this half
#pragma unroll 1
      for (int c0 = hf * 64; c0 < c_end; c0 += 16) {
        uint32_t r[16], pk[8];
        tmem_ld16(s_col + c0, r);
        tmem_wait_ld(r);
        if (c0 + 16 >= c_end) {   // all of S^T is in registers: its columns are free
          tc_fence_before();
          mbar_arrive(&sm.s_empty[slot]);
        }
        if (mode == kTimeOne)
          HSTU_QC_CHUNK(kTimeOne);
        else if (mode == kTimeTwo)
          HSTU_QC_CHUNK(kTimeTwo);
        else if (mode == kTimeFloat)
          HSTU_QC_CHUNK(kTimeFloat);
        else
          HSTU_QC_CHUNK(kTimeInt);
#pragma unroll
        for (int e = 0; e < 8; ++e) pk[e] = valid ? pk[e] : 0;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<uint4 *>(pt + (((((c0 & 63) >> 3) + e) ^ (key & 7)) << 4)) =
              make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
      }
#undef HSTU_QC_CHUNK
      fence_proxy_async_smem();   // P^T is written
      mbar_arrive(&sm.p_full[p_slot]);
      if constexpr (WEIGHTS) {
        if (j < sq.len && hf * 64 < nq)
          p.wpart[sq.wp0 + (int64_t(it.qtile * C::kHalves + hf) * H + h) * sq.len + j] =
              valid ? wsum : 0.f;
      }
    }
    // ---- O^T (lane = feature) through the P tiles' memory to rows of out ----
    const int c_first = w * 32, c_end = min(c_first + 32, nq);
    // The candidates' own v are fetched ahead of the last product: loaded behind it, 64
    // x 24 candidates on 512 keys took 57.8 us, so 52.3.
    uint4 vown[32 / kRows];
    const __nv_bfloat16 *v =
        static_cast<const __nv_bfloat16 *>(p.v) + q_row * p.v_rs + h * D + u * 8;
#pragma unroll
    for (int x = 0; x < 32 / kRows; ++x) {
      const int i = r0 + x * kRows;
      vown[x] = make_uint4(0, 0, 0, 0);
      if (it.split == 0 && i < nq) vown[x] = load_row8(v + i * p.v_rs, p.vec);
    }
    if (ok) ok = wait_cta_warp(&sm.o_full, 0, &sm.abort, p.wait);
    tc_fence_after();
    float *stage = reinterpret_cast<float *>(&sm.p[0][0]);   // [NQ][D]
    if (ok && quad * 32 < D) {
#pragma unroll 1
      for (int c0 = c_first; c0 < c_end; c0 += 16) {
        uint32_t r[16] = {};
        if (n_tiles > 0) {   // without a tile nothing has written O
          tmem_ld16(lanes + C::kO + c0, r);
          tmem_wait_ld(r);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) stage[(c0 + e) * D + key] = __uint_as_float(r[e]);
      }
    }
    named_bar_sync(3 + w, 128);
    if (ok) {
#pragma unroll
      for (int x = 0; x < 32 / kRows; ++x) {
        const int i = r0 + x * kRows;
        if (i >= c_end) break;
        const float4 oa = *reinterpret_cast<const float4 *>(stage + i * D + u * 8);
        const float4 ob = *reinterpret_cast<const float4 *>(stage + i * D + u * 8 + 4);
        float o[8] = {oa.x, oa.y, oa.z, oa.w, ob.x, ob.y, ob.z, ob.w};
        if (it.split == 0 && sm.own[i] != kQcNoOwn) {
          const uint32_t vs[4] = {vown[x].x, vown[x].y, vown[x].z, vown[x].w};
          const float own = sm.own[i];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            o[e] = fmaf(own, __uint_as_float(e & 1 ? vs[e / 2] & 0xFFFF0000u : vs[e / 2] << 16),
                        o[e]);
        }
        if (sq.splits > 1 || p.out_f32) {
          const float f = sq.splits > 1 ? 1.0f : p.scale;
          float *dst =
              sq.splits > 1
                  ? p.acc + ((sq.acc0 + (int64_t(it.split) * sq.n + i0 + i) * H + h) * D + u * 8)
                  : static_cast<float *>(p.out) + (q_row + i) * p.o_rs + h * D + u * 8;
          reinterpret_cast<float4 *>(dst)[0] =
              make_float4(o[0] * f, o[1] * f, o[2] * f, o[3] * f);
          reinterpret_cast<float4 *>(dst)[1] =
              make_float4(o[4] * f, o[5] * f, o[6] * f, o[7] * f);
        } else {
          __nv_bfloat16 *dst =
              static_cast<__nv_bfloat16 *>(p.out) + (q_row + i) * p.o_rs + h * D + u * 8;
          uint32_t ow[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            ow[e] = pack_bf16x2(o[2 * e] * p.scale, o[2 * e + 1] * p.scale);
          if (p.vec) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(ow[0], ow[1], ow[2], ow[3]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<uint16_t *>(dst)[e] = uint16_t(ow[e / 2] >> (16 * (e & 1)));
          }
        }
      }
    }
  } else {
    // ===================== decoding =====================
    const int dw = warp - 4 - C::kElemWarps;
    if (dw < C::kDecWarps)
      decode_tiles<D, NQ, false>(p, sm, it, sq, h, tmem, dw, lane);
    else
      decode_tiles<D, NQ, true>(p, sm, it, sq, h, tmem, dw - C::kDecWarps, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
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
