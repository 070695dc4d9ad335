// qcache_attn.cuh -- pieces shared by the attention kernels over the 4-bit
// cache and by their summing pass.
#pragma once

#include <math.h>

#include "qcache_host.h"

namespace hstu {

// A table entry below this hides its bucket: a pair in it adds exactly nothing,
// whatever its dot product and v are.  The kernels take such an entry as -inf, which a
// sum of two others never is, and leave out the pairs of a hidden bias.  NaN stays NaN.
constexpr float kQcBiasFloor = -1e30f;
constexpr float kQcHidden = -INFINITY;
__device__ __forceinline__ float qc_bias(float b) { return b < kQcBiasFloor ? kQcHidden : b; }
// SiLU of a candidate's own pair that is hidden: SiLU itself is never -inf.
constexpr float kQcNoOwn = -INFINITY;

// Where an item (blockIdx / heads) of the launch belongs.
struct QcItem {
  int seq, qtile, split;
  int32_t t0, t1;   // its 128-key tiles
};
__device__ __forceinline__ QcItem qc_item(const QcAttnParams &p, int item) {
  QcItem it;
  it.seq = qc_find(p.seqs, p.n_seqs, item, [](const QcAttnSeq &s) { return s.item0; });
  const QcAttnSeq &s = p.seqs[it.seq];
  const int x = item - s.item0;
  it.qtile = x / s.splits;
  it.split = x - it.qtile * s.splits;
  const int32_t tiles = (s.len + kQcKeyTile - 1) / kQcKeyTile;
  it.t0 = min(it.split * p.chunk, tiles);
  it.t1 = min(it.t0 + p.chunk, tiles);
  return it;
}

template <typename T>
__device__ __forceinline__ float qc_float(T x);
template <>
__device__ __forceinline__ float qc_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float qc_float<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T qc_round(float x);
template <>
__device__ __forceinline__ float qc_round<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 qc_round<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// N bytes global -> shared, zeros when !ok (src is then not read).
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src, bool ok) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src),
                 "r"(ok ? N : 0), "n"(N)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// 8 values of a bf16 row.
static __device__ __noinline__ uint4 load_row8_scalar(const __nv_bfloat16 *src) {
  uint32_t e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = reinterpret_cast<const uint16_t *>(src)[i];
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}
__device__ __forceinline__ uint4 load_row8(const __nv_bfloat16 *src, bool vec) {
  return vec ? *reinterpret_cast<const uint4 *>(src) : load_row8_scalar(src);
}
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// SiLU(x) = x / (1 + 2^y), y = -x log2 e, to a few 2^-22 of itself.
__device__ __forceinline__ float qc_silu(float x) {
  return x * rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * x));
}

}  // namespace hstu
