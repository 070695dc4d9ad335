// qcache.cu -- the 4-bit history cache: storing new rows (quantisation),
// reading rows back, and trimming a user's rows to the ones that received the
// most attention weight.  Format and rounding: qcache.cuh.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "qcache.cuh"
#include "qcache_host.h"

namespace hstu {
namespace qc {

// ---------------------------------------------------------------------------
// Append: quantise rows of K and V, write codes, parameters, time, position.
//
// Four consecutive lanes hold one group of 32 values (8 each), so a warp reads
// and writes consecutive addresses on both sides; the group's minimum and
// maximum take two shuffles.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;

// rne(x / s) of the exact quotient, given inv ~ 1 / s (to 2^-22): the product
// rounds to within one of it, and the remainder x - y s (exact in one fma)
// settles it.
__device__ __forceinline__ int rne_div(float x, float s, float inv) {
  const float y = rintf(x * inv);
  const float rem = fmaf(-y, s, x), half = 0.5f * s;
  const int i = int(y);
  const bool off = fabsf(rem) > half || (fabsf(rem) == half && (i & 1));
  return i + (off ? (rem > 0.f ? 1 : -1) : 0);
}

// The same where x has 8 significant bits (bf16) and s 4: x / s is then a tie
// between two integers or at least 2^-13 of its size away from one, so the
// float32 quotient (product and one correction) rounds to the integer that the
// exact one rounds to.  Adding 1.5 2^23 rounds to the nearest even integer.
__device__ __forceinline__ int rne_div_bf16(float x, float s, float inv) {
  const float q = x * inv;
  return __float_as_int(fmaf(fmaf(-q, s, x), inv, q) + 12582912.0f) - 0x4B400000;
}

// Scale of a group from its extremes, lo <= 0 <= hi: 4 significant bits.
__device__ __forceinline__ float group_scale(float lo, float hi) {
  // span = hi - lo exactly: rounded difference r plus its rounding error
  const float r = hi - lo, bb = r - hi, err = (hi - (r - bb)) + (-lo - bb);
  // r / 15 to within an ulp, truncated, is the scale or one step below it (a
  // product an ulp too large that reaches the next step reaches a scale that
  // 15 s >= span holds for); the exact 15 s decides
  float s = __uint_as_float(__float_as_uint(r * (1.0f / 15.0f)) & 0xFFF00000u);
  const float p = 15.0f * s;
  if (p < r || (p == r && err > 0.f)) s = __uint_as_float(__float_as_uint(s) + 0x00100000u);
  return fmaxf(s, 0x1p-126f);
}

__device__ __forceinline__ float held(float x) {   // NaN as 0, magnitudes to 2^126
  return x != x ? 0.f : fminf(fmaxf(x, -0x1p126f), 0x1p126f);
}

// Eight values as they come from memory, and their quantisation together with
// the 24 others of their group in the quad's other lanes.
template <typename T>
struct Eight;

template <>
struct Eight<float> {
  float x[8];
  __device__ __forceinline__ void load(const float *p, bool vec) {
    if (vec) {
      const float4 a = *reinterpret_cast<const float4 *>(p);
      const float4 b = *reinterpret_cast<const float4 *>(p + 4);
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = p[i];
    }
  }
  // This lane's extremes with 0; values brought into range.
  __device__ __forceinline__ void extremes(float &lo, float &hi) {
    lo = hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = held(x[i]);
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
    }
  }
  __device__ __forceinline__ float at(int i) const { return x[i]; }
  static __device__ __forceinline__ int rne(float x, float s, float inv) {
    return rne_div(x, s, inv);
  }
};

template <>
struct Eight<__nv_bfloat16> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, bool vec) {
    if (vec) {
      const uint4 a = *reinterpret_cast<const uint4 *>(p);
      w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = reinterpret_cast<const uint16_t *>(p)[2 * i] |
               uint32_t(reinterpret_cast<const uint16_t *>(p)[2 * i + 1]) << 16;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
  }
  __device__ __forceinline__ void extremes(float &lo, float &hi) {
    // two at a time; NaN and infinities show in them
    auto b2 = [](uint32_t v) { return *reinterpret_cast<const __nv_bfloat162 *>(&v); };
    const __nv_bfloat162 lo2 = __hmin2_nan(__hmin2_nan(b2(w[0]), b2(w[1])),
                                           __hmin2_nan(b2(w[2]), b2(w[3])));
    const __nv_bfloat162 hi2 = __hmax2_nan(__hmax2_nan(b2(w[0]), b2(w[1])),
                                           __hmax2_nan(b2(w[2]), b2(w[3])));
    lo = __bfloat162float(__hmin_nan(lo2.x, lo2.y));
    hi = __bfloat162float(__hmax_nan(hi2.x, hi2.y));
    if (!(lo >= -0x1p126f && hi <= 0x1p126f)) {   // rare: bring the values into range
      lo = hi = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = held(__uint_as_float(w[i] << 16));
        const float b = held(__uint_as_float(w[i] & 0xFFFF0000u));
        w[i] = (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xFFFF0000u);
        lo = fminf(lo, fminf(a, b));
        hi = fmaxf(hi, fmaxf(a, b));
      }
    }
    lo = fminf(lo, 0.f);
    hi = fmaxf(hi, 0.f);
  }
  static __device__ __forceinline__ int rne(float x, float s, float inv) {
    return rne_div_bf16(x, s, inv);
  }
};

// Codes and parameter of a group with extremes lo <= 0 <= hi, from this lane's
// eight values.  Zeros: s is at its floor, so z and the codes come out as 0.
template <typename T>
__device__ __forceinline__ void encode(const Eight<T> &x, float lo, float hi, uint32_t &word,
                                       uint32_t &param) {
  const float s = group_scale(lo, hi), inv = rcp_approx(s);
  const int z = Eight<T>::rne(-lo, s, inv);
  param = hi > lo ? (__float_as_uint(s) >> 16) | uint32_t(z) : 0u;
  word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    word |= uint32_t(min(Eight<T>::rne(x.at(i), s, inv) + z, 15)) << (4 * (i >> 1) + 16 * (i & 1));
}

// A unit is 8 values of one head's key or value row; `lanes` threads (a multiple
// of 4: a quad never straddles two tokens or two groups) share a token's units,
// keys first, then values.
struct RowThread {
  int64_t tok, row, pos;
  int u0;
  bool ok;
};
__device__ __forceinline__ RowThread row_thread(const QcRowsParams &p) {
  RowThread t;
  const int tpb = kRowThreads / p.lanes, tl = int(threadIdx.x) / p.lanes;
  t.u0 = int(threadIdx.x) - tl * p.lanes;
  t.tok = p.tok0 + int64_t(blockIdx.x) * tpb + tl;
  t.ok = tl < tpb && t.tok < p.tok_end;
  if (t.ok) {
    const int s = qc_find(p.seqs, p.n_seqs, t.tok, [](const QcRows &r) { return r.tok; });
    const int64_t i = t.tok - p.seqs[s].tok;
    t.row = p.seqs[s].row + i;
    t.pos = p.seqs[s].pos + i;
  }
  return t;
}
// Walks a thread's units of one operand: its place in the cache.  Where the lanes
// cover whole heads (64, 128, 256 values and 32) the next unit is a constant
// away; finding each by itself (a division, 64-bit products) cost as much as the
// quantisation.
template <bool IS_V>
struct UnitWalk {
  uint32_t *code;
  uint16_t *scale;
  int u;
  __device__ __forceinline__ static int words(const QCacheView &c) {   // per head and row
    return (IS_V ? c.d_v : c.d_qk) >> 3;
  }
  __device__ __forceinline__ UnitWalk(const QcRowsParams &p, int64_t row, int u_) : u(u_) {
    const QCacheView &c = p.cache;
    const int w = words(c);
    const int h = int(__umulhi(uint32_t(u * 8), IS_V ? p.v_magic : p.k_magic)), ew = u - h * w;
    const int64_t at = int64_t(h) * c.rows + row;
    code = (IS_V ? c.v_codes : c.k_codes) + (at * w + ew);
    scale = (IS_V ? c.v_scales : c.k_scales) + (at * (w >> 2) + (ew >> 2));
  }
  __device__ __forceinline__ void next(const QcRowsParams &p, int64_t row) {
    const int64_t step = IS_V ? p.v_step : p.k_step;   // heads x rows to the next unit, or 0
    u += p.lanes;
    if (step) {
      code += step * words(p.cache);
      scale += step * (words(p.cache) >> 2);
    } else {
      *this = UnitWalk(p, row, u);
    }
  }
};

// Bound by its instructions, about 180 per 32 lanes and unit (loads, extremes, scale,
// an exactly rounded quotient per value).  8 x 4,096 tokens, 8 heads of 128: 56 us,
// 172 MB (3.1 TB/s), issue slots 79 % busy.  Loading the next unit ahead, two units
// in flight and fewer warps with more registers took as long or longer.
template <typename T, bool IS_V>
__device__ __forceinline__ void append_units(const QcRowsParams &p, const RowThread &t) {
  const uint32_t quad = 0xFu << (threadIdx.x & 28);   // other quads may have left the loop
  const T *x0 = static_cast<const T *>(IS_V ? p.v : p.k) + t.tok * (IS_V ? p.v_rs : p.k_rs);
  UnitWalk<IS_V> w(p, t.row, t.u0);
  const int units = p.cache.heads * w.words(p.cache);
  for (; w.u < units; w.next(p, t.row)) {
    Eight<T> x;
    x.load(x0 + w.u * 8, p.vec);
    float lo, hi;
    x.extremes(lo, hi);
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(quad, lo, m));
      hi = fmaxf(hi, __shfl_xor_sync(quad, hi, m));
    }
    uint32_t word, param;
    encode<T>(x, lo, hi, word, param);
    *w.code = word;
    if ((w.u & 3) == 0) *w.scale = uint16_t(param);
  }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads, 6)
    append_kernel(const __grid_constant__ QcRowsParams p) {
  const RowThread t = row_thread(p);
  if (!t.ok) return;
  append_units<T, false>(p, t);
  append_units<T, true>(p, t);
  if (t.u0 == 0) {
    const QCacheView &c = p.cache;
    c.times[t.row] = p.ts[t.tok];
    c.pos[t.row] = int32_t(t.pos);
    if (c.weight) c.weight[t.row] = 0.f;
  }
}

// ---------------------------------------------------------------------------
// Read: the values that rows stand for, 8 per lane.  Of 8 x 4,096 rows, 8 heads of
// 128: 28 us, 172 MB (6.1 TB/s), near the memory's rate.
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void store_values(T *dst, uint32_t w, uint32_t param, bool vec) {
  if constexpr (sizeof(T) == 2) {
    uint32_t zz, ss, o[4];
    q4_group(param, zz, ss);
    q4_decode_bf16(w, zz, ss, o);
    if (vec) {
      *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        reinterpret_cast<uint16_t *>(dst)[i] = uint16_t(o[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    const float s = q4_scale(param);
    const int z = int(param & 15u);
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = s * float(q4_code(w, i) - z);
    if (vec) {
      reinterpret_cast<float4 *>(dst)[0] = make_float4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<float4 *>(dst)[1] = make_float4(o[4], o[5], o[6], o[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i] = o[i];
    }
  }
}

template <typename T, bool IS_V>
__device__ __forceinline__ void read_units(const QcRowsParams &p, const RowThread &t) {
  constexpr int N = 4;   // units in flight per thread
  T *row = static_cast<T *>(const_cast<void *>(IS_V ? p.v : p.k)) +
           t.tok * (IS_V ? p.v_rs : p.k_rs);
  UnitWalk<IS_V> at(p, t.row, t.u0);
  const int units = p.cache.heads * at.words(p.cache);
  while (at.u < units) {
    uint32_t w[N], par[N];
    const int u = at.u;
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (at.u < units) {
        w[k] = *at.code;
        par[k] = *at.scale;
        at.next(p, t.row);
      }
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (u + k * p.lanes < units)
        store_values<T>(row + (u + k * p.lanes) * 8, w[k], par[k], p.vec);
  }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    read_kernel(const __grid_constant__ QcRowsParams p) {
  const RowThread t = row_thread(p);
  if (!t.ok) return;
  read_units<T, false>(p, t);
  read_units<T, true>(p, t);
}

template <typename T, bool APPEND>
cudaError_t launch_rows_t(const QcRowsParams &p, cudaStream_t st) {
  const int tpb = kRowThreads / p.lanes;
  const int64_t blocks = (p.tok_end - p.tok0 + tpb - 1) / tpb;
  if (blocks <= 0) return cudaSuccess;
  if constexpr (APPEND)
    append_kernel<T><<<unsigned(blocks), kRowThreads, 0, st>>>(p);
  else
    read_kernel<T><<<unsigned(blocks), kRowThreads, 0, st>>>(p);
  count_launch();
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Eviction, step 1: which row every kept row comes from.
//
// One CTA per sequence.  A row's key is its weight as an ordered 32-bit
// integer, held in shared memory (up to kQcSelectKeys rows; recomputed from
// memory beyond).  The n-th largest key is found from its highest bits down; of
// the rows that share it the lowest are kept.  A kept row
// below n stays where it is; kept rows at or behind n fill the holes below n,
// both in ascending order, so the result does not depend on timing.
// Bound by latency: 16 rounds of one barrier, then five passes over the keys; 4,096
// rows 20 us, 32 sequences of up to 8,192 29 us.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

__device__ __forceinline__ uint32_t weight_key(float w, int32_t pos, int32_t keep_pos) {
  if (pos >= keep_pos) w = __int_as_float(0x7F800000);       // as if +inf
  if (w != w) w = -__int_as_float(0x7F800000);               // NaN as if -inf
  const uint32_t b = __float_as_uint(w + 0.0f);              // -0 and 0 are equal
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Exclusive sum over the block of one value per thread; *total gets the sum.
__device__ __forceinline__ uint32_t block_excl_sum(uint32_t v, uint32_t *warp_sums,
                                                   uint32_t *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // warp_sums may still be read from the call before
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  uint32_t s = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const uint32_t before = warp ? __shfl_sync(0xffffffffu, s, warp - 1) : 0u;
  return before + x - v;
}

__global__ void __launch_bounds__(kSelThreads)
    select_kernel(const __grid_constant__ QcEvictParams p) {
  extern __shared__ uint32_t keys[];     // [len] when it fits
  __shared__ uint32_t hist[256];
  __shared__ uint32_t warp_sums[kSelWarps];
  __shared__ uint32_t pick[2];           // chosen digit, keys above it
  const QcEvictSeq sq = p.seqs[blockIdx.x];
  const int tid = threadIdx.x, lane = tid & 31;
  const int32_t L = sq.len, n = sq.keep;
  int32_t *map = p.map + sq.map0;
  if (n >= L) {
    for (int32_t j = tid; j < n; j += kSelThreads) map[j] = j;
    return;
  }
  if (n == 0) return;
  const float *weight = p.src.weight + sq.row;
  const int32_t *pos = p.src.pos + sq.row;
  const bool cached = L <= p.key_cap;
  auto key_of = [&](int32_t j) {
    return cached ? keys[j] : weight_key(weight[j], pos[j], sq.keep_pos);
  };
  if (cached) {
    for (int32_t j = tid; j < L; j += kSelThreads)
      keys[j] = weight_key(weight[j], pos[j], sq.keep_pos);
  }
  // ---- the n-th largest key, and how many of its equals are kept (want) ----
  uint32_t prefix = 0, want = uint32_t(n);
  if (cached) {
    // Two bits at a time: count the keys at or above each of the three next
    // larger candidates.  16 rounds of a few compares per key and one barrier, with
    // three sets of counters: this round's, the last round's (still being read),
    // and the next one's (zero).
    if (tid < 9) hist[tid] = 0;
    uint32_t *cnt = hist, *next = hist + 3, *last = hist + 6;
    __syncthreads();   // keys and counters
    uint32_t above = 0;   // keys above the final prefix
    for (int shift = 30; shift >= 0; shift -= 2) {
      uint32_t c1 = 0, c2 = 0, c3 = 0;
      const uint32_t t1 = prefix | (1u << shift), t2 = prefix | (2u << shift),
                     t3 = prefix | (3u << shift);
      for (int32_t j = tid; j < L; j += kSelThreads) {
        const uint32_t k = keys[j];
        c1 += k >= t1;
        c2 += k >= t2;
        c3 += k >= t3;
      }
      c1 = __reduce_add_sync(0xffffffffu, c1);
      c2 = __reduce_add_sync(0xffffffffu, c2);
      c3 = __reduce_add_sync(0xffffffffu, c3);
      if (lane < 3) atomicAdd(&cnt[lane], lane == 0 ? c1 : lane == 1 ? c2 : c3);
      __syncthreads();
      const uint32_t a1 = cnt[0], a2 = cnt[1], a3 = cnt[2];
      // the largest candidate that at least n keys reach
      if (a3 >= uint32_t(n)) {
        prefix = t3;
      } else if (a2 >= uint32_t(n)) {
        prefix = t2;
        above = a3;
      } else if (a1 >= uint32_t(n)) {
        prefix = t1;
        above = a2;
      } else {
        above = a1;
      }
      // the last round's counters were read before this round's barrier
      if (tid < 3) last[tid] = 0;
      uint32_t *const spare = last;
      last = cnt;
      cnt = next;
      next = spare;
    }
    __syncthreads();   // the counters have been read: hist is free
    want = uint32_t(n) - above;
  } else {
    // Too long for shared memory: 8-bit digits, highest first, from a histogram.
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      for (int32_t j0 = 0; j0 < L; j0 += kSelThreads) {
        const int32_t j = j0 + tid;
        const uint32_t k = j < L ? key_of(j) : 0u;
        const bool in = j < L && (k & mask) == prefix;
        // equal digits of a warp are counted once (weights share exponents)
        const uint32_t d = in ? (k >> shift) & 255u : 256u + uint32_t(lane);
        const uint32_t same = __match_any_sync(0xffffffffu, d);
        if (in && lane == __ffs(same) - 1) atomicAdd(&hist[d], uint32_t(__popc(same)));
      }
      __syncthreads();
      // digits from 255 down: the one where the running count reaches want
      const uint32_t cnt = tid < 256 ? hist[255 - tid] : 0u;
      uint32_t total;
      const uint32_t before = block_excl_sum(cnt, warp_sums, &total);
      if (tid < 256 && before < want && before + cnt >= want) {
        pick[0] = uint32_t(255 - tid);
        pick[1] = before;
      }
      __syncthreads();
      prefix |= pick[0] << shift;
      want -= pick[1];
      __syncthreads();
    }
  }
  // ---- kept rows: every key above the threshold, and the first `want` at it ----
  // each thread owns a run of rows; an odd run length spreads the threads'
  // shared-memory accesses over the banks
  const int32_t run = ((L + kSelThreads - 1) / kSelThreads) | 1;
  const int32_t j0 = min(int64_t(tid) * run, int64_t(L)), j1 = min(int64_t(j0) + run, int64_t(L));
  uint32_t eq = 0, total;
  for (int32_t j = j0; j < j1; ++j) eq += key_of(j) == prefix;
  const uint32_t eq0 = block_excl_sum(eq, warp_sums, &total);
  uint32_t holes = 0, movers = 0, e = eq0;
  for (int32_t j = j0; j < j1; ++j) {
    const uint32_t k = key_of(j);
    const bool kept = k > prefix || (k == prefix && e++ < want);
    holes += !kept && j < n;
    movers += kept && j >= n;
  }
  const uint32_t hole0 = block_excl_sum(holes, warp_sums, &total);
  const uint32_t mover0 = block_excl_sum(movers, warp_sums, &total);
  int32_t *mov = p.movers + sq.map0;
  uint32_t m = mover0;
  e = eq0;
  for (int32_t j = j0; j < j1; ++j) {
    const uint32_t k = key_of(j);
    const bool kept = k > prefix || (k == prefix && e++ < want);
    if (kept && j >= n) mov[m++] = j;
    if (kept && j < n) map[j] = j;
  }
  __syncthreads();   // the movers' list is complete (same block reads it below)
  uint32_t hl = hole0;
  e = eq0;
  for (int32_t j = j0; j < min(j1, n); ++j) {
    const uint32_t k = key_of(j);
    const bool kept = k > prefix || (k == prefix && e++ < want);
    if (!kept) map[j] = mov[hl++];
  }
}

// ---------------------------------------------------------------------------
// Eviction, step 2: copy the rows.  A unit is one group (16 bytes of codes and
// its parameter); consecutive lanes write consecutive groups.  In place only
// the holes are written, and every source lies at or behind `keep`.  Bound by
// latency of scattered 16-byte reads: halving 32 histories of 1,024 to 8,192 rows, 8
// heads of 128, takes 25 us, with 116 MB at the memory (4.6 TB/s).
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kMoveUnits = 2;   // 1 and 4: a microsecond or two longer, 8: four

__global__ void __launch_bounds__(kMoveThreads)
    move_kernel(const __grid_constant__ QcEvictParams p) {
  const int sqi = qc_find(p.seqs, p.n_seqs, int64_t(blockIdx.x),
                          [](const QcEvictSeq &s) { return s.block0; });
  const QcEvictSeq sq = p.seqs[sqi];
  const QCacheView &a = p.src, &b = p.dst;
  const int64_t r0 = (int64_t(blockIdx.x) - sq.block0) * p.move_rows;
  const int rows = int(min(int64_t(p.move_rows), int64_t(sq.keep) - r0));
  const int32_t *map = p.map + sq.map0 + r0;
  for (int r = threadIdx.x; r < rows; r += kMoveThreads) {
    const int32_t m = map[r];
    if (p.in_place && m == r0 + r) continue;
    b.times[sq.dst_row + r0 + r] = a.times[sq.row + m];
    b.pos[sq.dst_row + r0 + r] = a.pos[sq.row + m];
    b.weight[sq.dst_row + r0 + r] = a.weight[sq.row + m];
  }
  const int gk = a.d_qk >> 5, gv = a.d_v >> 5;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    const int gs = part ? gv : gk;
    const uint4 *ac = reinterpret_cast<const uint4 *>(part ? a.v_codes : a.k_codes);
    uint4 *bc = reinterpret_cast<uint4 *>(part ? b.v_codes : b.k_codes);
    const uint16_t *as = part ? a.v_scales : a.k_scales;
    uint16_t *bs = part ? b.v_scales : b.k_scales;
    const int per_head = rows * gs, all = per_head * a.heads;
    // kMoveUnits groups in flight per thread
#pragma unroll 1
    for (int x0 = threadIdx.x; x0 < all; x0 += kMoveUnits * kMoveThreads) {
      int64_t to[kMoveUnits];
      uint4 code[kMoveUnits];
      uint16_t par[kMoveUnits];
#pragma unroll
      for (int k = 0; k < kMoveUnits; ++k) {
        const int x = x0 + k * kMoveThreads;
        to[k] = -1;
        if (x < all) {
          const int h = x / per_head, y = x - h * per_head, r = y / gs, g = y - r * gs;
          const int32_t m = map[r];
          if (!(p.in_place && m == r0 + r)) {
            const int64_t from = (int64_t(h) * a.rows + sq.row + m) * gs + g;
            to[k] = (int64_t(h) * b.rows + sq.dst_row + r0 + r) * gs + g;
            code[k] = ac[from];
            par[k] = as[from];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kMoveUnits; ++k)
        if (to[k] >= 0) {
          bc[to[k]] = code[k];
          bs[to[k]] = par[k];
        }
    }
  }
}

}  // namespace qc

cudaError_t launch_qcache_append(const QcRowsParams &p, bool bf16, cudaStream_t st) {
  return bf16 ? qc::launch_rows_t<__nv_bfloat16, true>(p, st)
              : qc::launch_rows_t<float, true>(p, st);
}
cudaError_t launch_qcache_read(const QcRowsParams &p, bool bf16, cudaStream_t st) {
  return bf16 ? qc::launch_rows_t<__nv_bfloat16, false>(p, st)
              : qc::launch_rows_t<float, false>(p, st);
}

cudaError_t launch_qcache_evict(const QcEvictParams &p, int32_t max_len, int64_t move_blocks,
                                cudaStream_t st) {
  using namespace qc;
  static PerDeviceOnce attr;
  cudaError_t e = set_smem_once(attr, select_kernel, kQcSelectKeys * sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  const int32_t keys = max_len < kQcSelectKeys ? max_len : kQcSelectKeys;
  QcEvictParams q = p;
  q.key_cap = keys;
  select_kernel<<<unsigned(p.n_seqs), kSelThreads, size_t(keys) * sizeof(uint32_t), st>>>(q);
  count_launch();
  e = cudaGetLastError();
  if (e != cudaSuccess || move_blocks == 0) return e;
  move_kernel<<<unsigned(move_blocks), kMoveThreads, 0, st>>>(q);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hstu
