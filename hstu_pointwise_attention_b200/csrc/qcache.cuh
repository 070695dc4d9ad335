// qcache.cuh -- the 4-bit history cache: its number format and the per-call
// tables its kernels share.
//
// Format.  Groups of 32 consecutive values of one head's row share a scale s
// and a zero point z; a value is s (q - z) with q in 0..15.  The keys and
// values of the HSTU layer are SiLU outputs (>= -0.28, open above), so a grid
// symmetric about zero would leave nearly half its codes unused; the zero point
// costs four bits per group.  s has 4 significant bits: |q - z| <= 15 has 4, so
// every stored value has at most 8 significant bits and is exact in bfloat16,
// and the tensor cores multiply exactly the stored values.
//   lo = min(0, min x), hi = max(0, max x) over the group
//   s  = the smallest float with 4 significant bits, s >= 2^-126, 15 s >= hi - lo
//   z  = rne(-lo / s),  q = clamp(rne(x / s) + z, 0, 15)   (exact quotients)
// A group of zeros has s = 0, z = 0, q = 0.  NaN is stored as 0 and magnitudes
// are held to 2^126 (infinities among them).  The 16-bit parameter is the upper
// 12 bits of s as a bfloat16 (its low 4 mantissa bits are zero) with z in the
// low 4 bits.  Eight codes make one 32-bit word: nibble i holds element 2 i,
// nibble i + 4 element 2 i + 1, so (w >> 4 i) & 0x000F000F is the pair of codes
// (2 i, 2 i + 1) in the halves of a register.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace hstu {

// Device pointers of one cache (include/hstu.h, hstu_qcache_t).
struct QCacheView {
  int64_t rows;
  int32_t heads, d_qk, d_v;
  uint32_t *k_codes, *v_codes;     // [H][rows][d / 8] words of 8 codes
  uint16_t *k_scales, *v_scales;   // [H][rows][d / 32]
  int64_t *times;                  // [rows]
  int32_t *pos;                    // [rows]
  float *weight;                   // [rows], may be null
};

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Sequences per launch: their table travels in the kernel's parameters, so a
// call needs no upload and records whole under stream capture.
constexpr int kQcMaxSeqs = 64;

// The last sequence of table t[0..n) whose `first` is <= x (first is
// non-decreasing and t[0].first = 0 <= x).
template <class T, class I, class F>
__device__ __forceinline__ int qc_find(const T *t, int n, I x, F first) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (I(first(t[mid])) <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// ---- decoding ----
__device__ __forceinline__ float q4_scale(uint32_t param) {
  return __uint_as_float((param & 0xFFF0u) << 16);
}

// (x & mask) | bits as one instruction: written as two operations on constants,
// it compiled to two (the attention of 64 single events took 98 us instead of 88).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));
  return y;
}
// The 8 values of one word as 4 bfloat16 pairs, exact: 0x4300 | q is the
// bfloat16 128 + q, minus 128 + z leaves q - z (both exact), times s (exact,
// see above).
__device__ __forceinline__ void q4_decode_bf16(uint32_t w, uint32_t zz, uint32_t ss,
                                               uint32_t (&out)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = and_or(w >> (4 * i), 0x000F000Fu, 0x43004300u);
    __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162 *>(&m);
    x = __hsub2(x, *reinterpret_cast<const __nv_bfloat162 *>(&zz));
    x = __hmul2(x, *reinterpret_cast<const __nv_bfloat162 *>(&ss));
    out[i] = *reinterpret_cast<const uint32_t *>(&x);
  }
}
// The group's operands of q4_decode_bf16, 128 + z and s; `pair` holds the parameters
// of the two values of a pair (twice the same, or those of two rows).
__device__ __forceinline__ void q4_group_pair(uint32_t pair, uint32_t &zz, uint32_t &ss) {
  zz = and_or(pair, 0x000F000Fu, 0x43004300u);
  ss = pair & 0xFFF0FFF0u;
}
__device__ __forceinline__ void q4_group(uint32_t param, uint32_t &zz, uint32_t &ss) {
  q4_group_pair(__byte_perm(param, 0, 0x1010), zz, ss);
}
// Code of element e (0..7) of a word.
__device__ __forceinline__ int q4_code(uint32_t w, int e) {
  return int((w >> (4 * (e >> 1) + 16 * (e & 1))) & 15u);
}

}  // namespace hstu
