// qcache_attn_few.cu -- up to 8 candidates against the 4-bit history cache
// (single events above all), bf16, d_qk = d_v in {64, 128}.
//
//   out_i = c (sum_j SiLU(x_ij) v_j + SiLU(x_ii) v_i),
//   x_ij = alpha <q_i, k_j> + rab_pos[P_b - pos_j] + rab_time[tb(t_i - t_j)]
//   w_j  <- decay w_j + c sum_{i, h} |SiLU(x_ij)|
//
// With few candidates the work is the reading and decoding of the cache, and the
// products are small: S^T = K Q^T and O^T += V^T P^T by warp-level m16n8k16
// MMAs, 16 keys (16 features of V) x 8 candidates.  Their A operand is registers,
// so a decoded value goes straight into the product; through the tcgen05 unit it
// would be written to shared or tensor memory and read back, and the tile of at
// least 64 x 128 pairs would be nearly all padding.
//
// One CTA = (sequence, head, 8 candidates, range of 128-key tiles), 4 warps that
// take 32 keys by turns.  A warp copies its own codes (cp.async, two stages) and
// shares nothing with the others until the end, so the loop has no barrier but
// the warp's.  The order of the keys within a step and of the features within a
// product is free, as long as both operands use the same:
//   K: lane (g, t) = (lane / 4, lane % 4) takes word t of each group of 32, keys
//      key_of(g) and 8 + key_of(g); a word's four pairs of codes are the lane's
//      share of two k16 products.
//   V: the lane takes words (D / 64) g .. of keys t, 4 + t, 8 + t, 12 + t; a code
//      of two keys side by side is one operand register, so that one product has
//      features 2 i of the words in rows 0-7 and 2 i + 1 in rows 8-15.
//   P^T goes from the accumulators of the first product to the B operand of the
//      second by two 8 x 8 transpositions.
// The row permutation key_of (2 t + e -> t + 4 e) and the chunk swizzles below make
// both reads of a stage free of bank conflicts.
//
// Bound by instructions: about 1,040 per 32 keys of 128, half of them decoding.  Measured
// (64 histories of 1,024 to 8,192 events, one candidate each, 8 heads of 128, weights
// updated): 81 us and 7 more to sum, 237 MB, 2.8 TB/s; issue slots 67 % busy, integer
// unit 60 %.  The 64-wide tcgen05 tiles take 155 us there.  Two or eight warps per CTA
// take 5 to 10 us longer, a third stage or four chains of products change nothing.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "qcache_attn.cuh"
#include "tile_common.cuh"

namespace hstu {
namespace qc_few {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kQ = kQcFewQueries;
constexpr int kKeys = 32;      // per warp and step
constexpr int kStages = 2;

template <int D>
struct Stage {
  alignas(16) uint8_t k[kKeys * D / 2];
  alignas(16) uint8_t v[kKeys * D / 2];
  alignas(16) uint16_t ks[kKeys * D / 32];
  alignas(16) uint16_t vs[kKeys * D / 32];
};
template <int D>
struct Smem {
  union {
    Stage<D> st[kWarps][kStages];
    float o[kWarps][kQ][D + 4];    // the warps' sums, at the end
  };
  float own[kQ];                   // SiLU of the candidates' own pairs
};

__device__ __forceinline__ int key_of(int r) { return (r >> 1) + 4 * (r & 1); }
// Place of 16-byte chunk c of a key's row.
template <int D>
__device__ __forceinline__ int k_chunk(int key, int c) {
  return key * (D / 2) + ((D == 128 ? c ^ ((key >> 1) & 3) : c ^ ((key >> 2) & 1)) << 4);
}
template <int D>
__device__ __forceinline__ int v_chunk(int key, int c) {
  return key * (D / 2) + ((D == 128 ? c ^ (key & 2) : c) << 4);
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 4)
    attn_kernel(const __grid_constant__ QcAttnParams p) {
  extern __shared__ float4 sm4[];
  Smem<D> &sm = *reinterpret_cast<Smem<D> *>(sm4);
  constexpr int G = D / 32, W = D / 64;   // groups of a row; V words per lane and key
  const QCacheView &cv = p.cache;
  const int H = cv.heads;
  const int item = int(blockIdx.x) / H, h = int(blockIdx.x) - item * H;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (p.clear_err && blockIdx.x == 0 && tid < 4) p.wait.err[tid] = 0;
  const QcItem it = qc_item(p, item);
  const QcAttnSeq &sq = p.seqs[it.seq];
  const int nq = min(kQ, sq.n - it.qtile * kQ);
  const int64_t q_row = sq.q0 + it.qtile * kQ;
  const float *rp = p.rab_p + (p.rab_per_head ? int64_t(h) * p.nb_p : 0);
  const float *rt = p.rab_t + (p.rab_per_head ? int64_t(h) * p.nb_t : 0);

  // ---- the warp's copies ----
  // Copy u of a step is the lane's chunk (u * 32 + lane) of its K (or V) codes.  All
  // copies of a lane have the same swizzle, so each is a constant away from the first.
  const int32_t j_end = min(it.t1 * kQcKeyTile, sq.len);
  int32_t jb = it.t0 * kQcKeyTile + warp * kKeys;   // first key of the step
  const uint32_t st0 = smem_u32(&sm.st[warp][0]);
  const uint32_t k_dst = k_chunk<D>(lane / G, lane % G), v_dst = v_chunk<D>(lane / G, lane % G);
  const int64_t at0 = int64_t(h) * cv.rows + sq.row;
  const uint8_t *k_src = reinterpret_cast<const uint8_t *>(cv.k_codes) + (at0 + jb) * (D / 2) + lane * 16;
  const uint8_t *v_src = reinterpret_cast<const uint8_t *>(cv.v_codes) + (at0 + jb) * (D / 2) + lane * 16;
  const uint16_t *ks_src = cv.k_scales + (at0 + jb + lane) * G;
  const uint16_t *vs_src = cv.v_scales + (at0 + jb + lane) * G;
  int32_t j_copy = jb;
  auto copy = [&](uint32_t st) {   // keys [j_copy, j_copy + 32) of the cache, zeros from j_end on
    const int32_t left = j_end - j_copy;
    if (left >= kKeys) {
#pragma unroll
      for (int u = 0; u < G; ++u) {
        cp_async<16>(st + offsetof(Stage<D>, k) + k_dst + u * 512, k_src + u * 512, true);
        cp_async<16>(st + offsetof(Stage<D>, v) + v_dst + u * 512, v_src + u * 512, true);
      }
      cp_async<2 * G>(st + offsetof(Stage<D>, ks) + lane * 2 * G, ks_src, true);
      cp_async<2 * G>(st + offsetof(Stage<D>, vs) + lane * 2 * G, vs_src, true);
    } else if (left > 0) {
#pragma unroll 1
      for (int u = 0; u < G; ++u) {
        const bool ok = u * (32 / G) + lane / G < left;
        cp_async<16>(st + offsetof(Stage<D>, k) + k_dst + u * 512,
                     ok ? k_src + u * 512 : reinterpret_cast<const uint8_t *>(cv.k_codes), ok);
        cp_async<16>(st + offsetof(Stage<D>, v) + v_dst + u * 512,
                     ok ? v_src + u * 512 : reinterpret_cast<const uint8_t *>(cv.v_codes), ok);
      }
      const bool ok = lane < left;
      cp_async<2 * G>(st + offsetof(Stage<D>, ks) + lane * 2 * G, ok ? ks_src : cv.k_scales, ok);
      cp_async<2 * G>(st + offsetof(Stage<D>, vs) + lane * 2 * G, ok ? vs_src : cv.v_scales, ok);
    }
    cp_async_commit();
    j_copy += kWarps * kKeys;
    k_src += kWarps * kKeys * D / 2;
    v_src += kWarps * kKeys * D / 2;
    ks_src += kWarps * kKeys * G;
    vs_src += kWarps * kKeys * G;
  };
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) copy(st0 + s * uint32_t(sizeof(Stage<D>)));

  // ---- the candidates ----
  uint32_t bq[G][4];
  {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + (q_row + g) * p.q_rs +
                             int64_t(h) * D + 8 * t;
#pragma unroll
    for (int u = 0; u < G; ++u) {
      const uint4 w = g < nq ? load_row8(q + 32 * u, p.vec) : make_uint4(0, 0, 0, 0);
      bq[u][0] = w.x;
      bq[u][1] = w.y;
      bq[u][2] = w.z;
      bq[u][3] = w.w;
    }
  }
  // the times of the lane's two candidates; `one_time`: all of them are the same
  const int64_t t_first = p.cand_ts[q_row];
  const int64_t tq0 = 2 * t < nq ? p.cand_ts[q_row + 2 * t] : t_first;
  const int64_t tq1 = 2 * t + 1 < nq ? p.cand_ts[q_row + 2 * t + 1] : t_first;
  const bool one_time = __all_sync(0xffffffffu, tq0 == t_first && tq1 == t_first);
  const bool live0 = 2 * t < nq, live1 = 2 * t + 1 < nq;
  float *wp = p.weight_rows > 0
                  ? p.wpart + sq.wp0 + (int64_t(it.qtile) * H + h) * sq.len
                  : nullptr;

  // the candidates' own pairs (distance 0 in position and time)
  if (it.split == 0) {
    for (int i = warp; i < nq; i += kWarps) {
      const __nv_bfloat16 *qr =
          static_cast<const __nv_bfloat16 *>(p.q) + (q_row + i) * p.q_rs + int64_t(h) * D;
      const __nv_bfloat16 *kr =
          static_cast<const __nv_bfloat16 *>(p.k) + (q_row + i) * p.k_rs + int64_t(h) * D;
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < D; e += 32)
        dot = fmaf(__bfloat162float(qr[e + lane]), __bfloat162float(kr[e + lane]), dot);
#pragma unroll
      for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
      const float b = qc_bias(rp[0]) + qc_bias(rt[0]);
      if (lane == 0) sm.own[i] = b == kQcHidden ? kQcNoOwn : qc_silu(fmaf(p.alpha, dot, b));
    }
  } else if (tid < kQ) {
    sm.own[tid] = kQcNoOwn;
  }

  float o[4 * W][4];
#pragma unroll
  for (int m = 0; m < 4 * W; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[m][e] = 0.f;

  // position and time of key jb + lane, loaded a step ahead
  int32_t kp = 0;
  int64_t kt = 0;
  auto load_key = [&](int32_t j) {
    const int64_t r = sq.row + min(j + lane, j_end - 1);
    kp = cv.pos[r];
    kt = cv.times[r];
  };
  if (jb < j_end) load_key(jb);
  // where the lane reads in a stage (the swizzles repeat every 8 keys)
  const int ka0 = key_of(g);
  uint32_t k_at[G];
#pragma unroll
  for (int u = 0; u < G; ++u) k_at[u] = k_chunk<D>(ka0, u) + 4 * t;
  const uint32_t v_at = v_chunk<D>(t, (W * g) >> 2) + ((W * g) & 3) * 4;
  const uint32_t vs_at = (t * G + ((W * g) >> 2)) * 2;
  int cur = 0;
#pragma unroll 1
  for (; jb < j_end; jb += kWarps * kKeys) {
    // the key's bias, with the time's where all candidates share it
    const int64_t tk = kt;
    float bias = qc_bias(rp[pos_bucket(int64_t(sq.pos) - kp, p.nb_p)]);
    if (one_time) bias += qc_bias(rt[time_bucket_i64(t_first - tk, p.sub_bits, p.nb_t)]);
    if (jb + kWarps * kKeys < j_end) load_key(jb + kWarps * kKeys);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const Stage<D> &st = sm.st[warp][cur];
    const uint8_t *const k_base = st.k;
    const uint8_t *kw[G];
#pragma unroll
    for (int u = 0; u < G; ++u) kw[u] = k_base + k_at[u];
    const uint8_t *const vw = st.v + v_at;
    const uint8_t *const kpar = reinterpret_cast<const uint8_t *>(st.ks) + ka0 * 2 * G;
    const uint8_t *const vpar = reinterpret_cast<const uint8_t *>(st.vs) + vs_at;
#pragma unroll
    for (int r0 = 0; r0 < kKeys; r0 += 16) {
      // ---- S^T = K Q^T: keys ka, kb = ka + 8 of this lane ----
      const int ka = r0 + ka0, kb = ka + 8;
      float s[2][4] = {};
      uint32_t pa[(G + 1) / 2], pb[(G + 1) / 2];
      if constexpr (G == 4) {
        const uint2 a = *reinterpret_cast<const uint2 *>(kpar + r0 * 2 * G);
        const uint2 b = *reinterpret_cast<const uint2 *>(kpar + (r0 + 8) * 2 * G);
        pa[0] = a.x, pa[1] = a.y, pb[0] = b.x, pb[1] = b.y;
      } else {
        pa[0] = *reinterpret_cast<const uint32_t *>(kpar + r0 * 2 * G);
        pb[0] = *reinterpret_cast<const uint32_t *>(kpar + (r0 + 8) * 2 * G);
      }
#pragma unroll
      for (int u = 0; u < G; ++u) {
        const uint32_t wa = *reinterpret_cast<const uint32_t *>(kw[u] + r0 * (D / 2));
        const uint32_t wb = *reinterpret_cast<const uint32_t *>(kw[u] + (r0 + 8) * (D / 2));
        const uint32_t da = __byte_perm(pa[u / 2], 0, u & 1 ? 0x3232 : 0x1010);
        const uint32_t db = __byte_perm(pb[u / 2], 0, u & 1 ? 0x3232 : 0x1010);
        uint32_t xa[4], xb[4], zz, ss;
        q4_group_pair(da, zz, ss);
        q4_decode_bf16(wa, zz, ss, xa);
        q4_group_pair(db, zz, ss);
        q4_decode_bf16(wb, zz, ss, xb);
        mma(s[0], xa[0], xb[0], xa[1], xb[1], bq[u][0], bq[u][1]);
        mma(s[1], xa[2], xb[2], xa[3], xb[3], bq[u][2], bq[u][3]);
      }
      // ---- P = SiLU(x): (ka, 2t), (ka, 2t + 1), (kb, 2t), (kb, 2t + 1) ----
      float ca = __shfl_sync(0xffffffffu, bias, ka), cb = __shfl_sync(0xffffffffu, bias, kb);
      float b[4] = {ca, ca, cb, cb};
      if (!one_time) {
        const int64_t ta = __shfl_sync(0xffffffffu, (long long)tk, ka);
        const int64_t tb = __shfl_sync(0xffffffffu, (long long)tk, kb);
        b[0] += qc_bias(rt[time_bucket_i64(tq0 - ta, p.sub_bits, p.nb_t)]);
        b[1] += qc_bias(rt[time_bucket_i64(tq1 - ta, p.sub_bits, p.nb_t)]);
        b[2] += qc_bias(rt[time_bucket_i64(tq0 - tb, p.sub_bits, p.nb_t)]);
        b[3] += qc_bias(rt[time_bucket_i64(tq1 - tb, p.sub_bits, p.nb_t)]);
      }
      const bool ok_a = jb + ka < j_end, ok_b = jb + kb < j_end;
      float pv[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = qc_silu(fmaf(p.alpha, s[0][e] + s[1][e], b[e]));
        pv[e] = (e < 2 ? ok_a : ok_b) && b[e] != kQcHidden ? x : 0.f;
      }
      if (wp) {
        float w0 = (live0 ? fabsf(pv[0]) : 0.f) + (live1 ? fabsf(pv[1]) : 0.f);
        float w1 = (live0 ? fabsf(pv[2]) : 0.f) + (live1 ? fabsf(pv[3]) : 0.f);
        w0 += __shfl_xor_sync(0xffffffffu, w0, 1);
        w1 += __shfl_xor_sync(0xffffffffu, w1, 1);
        w0 += __shfl_xor_sync(0xffffffffu, w0, 2);
        w1 += __shfl_xor_sync(0xffffffffu, w1, 2);
        if (t == 0 && ok_a) wp[jb + ka] = w0;
        if (t == 0 && ok_b) wp[jb + kb] = w1;
      }
      const uint32_t b0 = transpose8(pack_bf16x2(pv[0], pv[1]));
      const uint32_t b1 = transpose8(pack_bf16x2(pv[2], pv[3]));
      // ---- O^T += V^T P^T: keys t, 4 + t (a0, a1) and 8 + t, 12 + t (a2, a3) ----
      uint32_t w[4][W], zz[2], ss[2];
      uint32_t par[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint8_t *src = vw + (r0 + 4 * e) * (D / 2);
        if constexpr (W == 2) {
          const uint2 x = *reinterpret_cast<const uint2 *>(src);
          w[e][0] = x.x, w[e][1] = x.y;
        } else {
          w[e][0] = *reinterpret_cast<const uint32_t *>(src);
        }
        par[e] = *reinterpret_cast<const uint16_t *>(vpar + (r0 + 4 * e) * 2 * G);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
        q4_group_pair(__byte_perm(par[2 * e], par[2 * e + 1], 0x5410), zz[e], ss[e]);
#pragma unroll
      for (int x = 0; x < W; ++x) {
        uint32_t a[4][4];   // features 2 i (a[0], a[2]) and 2 i + 1 of the key pairs
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          q4_decode_bf16(__byte_perm(w[2 * e][x], w[2 * e + 1][x], 0x5410), zz[e], ss[e],
                         a[2 * e]);
          q4_decode_bf16(__byte_perm(w[2 * e][x], w[2 * e + 1][x], 0x7632), zz[e], ss[e],
                         a[2 * e + 1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mma(o[x * 4 + i], a[0][i], a[1][i], a[2][i], a[3][i], b0, b1);
      }
    }
    __syncwarp();   // the warp has read the stage
    copy(st0 + cur * uint32_t(sizeof(Stage<D>)));
    cur ^= 1;
  }
  cp_async_wait<0>();
  __syncthreads();   // the stages become the warps' sums
#pragma unroll
  for (int x = 0; x < W; ++x)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 8 * (W * g + x) + 2 * i;
      *reinterpret_cast<float2 *>(&sm.o[warp][2 * t][e]) =
          make_float2(o[x * 4 + i][0], o[x * 4 + i][2]);
      *reinterpret_cast<float2 *>(&sm.o[warp][2 * t + 1][e]) =
          make_float2(o[x * 4 + i][1], o[x * 4 + i][3]);
    }
  __syncthreads();
  for (int x = tid; x < nq * D; x += kThreads) {
    const int i = x / D, e = x % D;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += sm.o[w][i][e];
    const int64_t row = q_row + i;
    if (sm.own[i] != kQcNoOwn)
      sum = fmaf(sm.own[i],
                 __bfloat162float(
                     static_cast<const __nv_bfloat16 *>(p.v)[row * p.v_rs + int64_t(h) * D + e]),
                 sum);
    if (sq.splits > 1)
      p.acc[(sq.acc0 + (int64_t(it.split) * sq.n + it.qtile * kQ + i) * H + h) * D + e] = sum;
    else if (p.out_f32)
      static_cast<float *>(p.out)[row * p.o_rs + int64_t(h) * D + e] = sum * p.scale;
    else
      static_cast<__nv_bfloat16 *>(p.out)[row * p.o_rs + int64_t(h) * D + e] =
          __float2bfloat16_rn(sum * p.scale);
  }
}

}  // namespace qc_few

cudaError_t launch_qcache_attn_few(const QcAttnParams &p, cudaStream_t st) {
  using namespace qc_few;
  static PerDeviceOnce attr64, attr128;
  const bool wide = p.cache.d_qk == 128;
  const size_t smem = wide ? sizeof(Smem<128>) : sizeof(Smem<64>);
  const cudaError_t e = wide ? set_smem_once(attr128, attn_kernel<128>, smem)
                             : set_smem_once(attr64, attn_kernel<64>, smem);
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(p.items) * unsigned(p.cache.heads);
  if (wide)
    attn_kernel<128><<<grid, kThreads, smem, st>>>(p);
  else
    attn_kernel<64><<<grid, kThreads, smem, st>>>(p);
  count_launch();
  return cudaGetLastError();
}

}  // namespace hstu
