// qcache_attn.cuh -- pieces shared by the attention kernels over the 4-bit
// cache (CUDA-core and tensor-core) and by their summing pass.
#pragma once

#include "qcache_host.h"

namespace hstu {

// SiLU(x) = x / (1 + e^-x), 0 in the limit x -> -inf: the kernels keep the
// bias of a logit at or above this, so a table entry of -inf or of the lowest
// float hides its bucket instead of giving -inf * 0.  NaN stays NaN.
constexpr float kQcBiasFloor = -1e30f;
__device__ __forceinline__ float qc_bias(float b) { return b < kQcBiasFloor ? kQcBiasFloor : b; }

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

}  // namespace hstu
