// qcache_host.h -- launch parameters of the 4-bit cache kernels, filled by
// qcache_api.cu.  Each holds the table of up to kQcMaxSeqs sequences by value
// (kernel parameters, at most 8 KB), so no call uploads anything.
#pragma once

#include "internal.h"
#include "qcache.cuh"

namespace hstu {

// Rows (or candidates) of one sequence: the kernels' loops step int32 indices by up
// to 1,024 and round lengths up to tiles.
constexpr int64_t kQcMaxLen = (int64_t(1) << 31) - 1024;

// --- append / read ---
// From this many tokens on 32 threads share a token, which spares instructions
// (8 heads of 128, 8 x 4096 tokens stored and read: 85 us, 64 threads 99, 128
// threads 132); below, 128, which take fewer steps (8 x 1 tokens: 5.6 us, 32 threads
// 8.6).  3,840 rows read: 32 threads 2 us faster than 128.
constexpr int kQcManyRows = 2048;
struct QcRows {
  int64_t tok;     // first token (row of k, v)
  int64_t row;     // its cache row
  int64_t pos;     // its position (append)
};
struct QcRowsParams {
  QCacheView cache;
  const void *k, *v;       // activations; read_kernel writes them
  int64_t k_rs, v_rs;
  const int64_t *ts;       // append
  int64_t tok0, tok_end;   // tokens of this launch
  uint32_t k_magic, v_magic;   // 2^32 / d, rounded up: element / d for element < 2^20
  int64_t k_step, v_step;      // cache rows from a thread's unit to its next, 0: not constant
  int32_t lanes;               // threads per token
  int32_t n_seqs;
  bool vec;                // 16-byte accesses to k and v are aligned
  QcRows seqs[kQcMaxSeqs];
};

// --- evict ---
constexpr int kQcSelectKeys = 40 * 1024; // keys the selection holds in shared memory
struct QcEvictSeq {
  int64_t row, dst_row;
  int64_t map0;            // first entry of the sequence in map / movers
  int64_t block0;          // first block of its copy
  int32_t len, keep, keep_pos, pad;
};
struct QcEvictParams {
  QCacheView src, dst;
  int32_t *map, *movers;
  int32_t n_seqs, key_cap;
  int32_t move_rows;       // kept rows per block of the copy
  bool in_place;
  QcEvictSeq seqs[kQcMaxSeqs];
};

// --- attention over the cache ---
struct QcAttnSeq {
  int64_t row, q0;         // first cache row, first candidate row
  int64_t acc0;            // first row of its partial outputs [split][n][H]
  int64_t wp0;             // first float of its weight partials [plane][H][len]
  int64_t wrow0;           // its first row in the weight pass of this launch
  int32_t len, n, pos;     // cached rows, candidates, the candidates' position
  int32_t item0;           // its first item (query tile x key range) in this launch
  int32_t splits, fin0;    // key ranges; its first row in the summing pass
};
struct QcAttnParams {
  QCacheView cache;
  const void *q, *k, *v;
  void *out;
  int64_t q_rs, k_rs, v_rs, o_rs;
  const int64_t *cand_ts;
  const float *rab_p, *rab_t;
  float *acc, *wpart;
  WaitCtl wait;
  float alpha, scale, decay;
  int32_t nb_p, nb_t, sub_bits;
  int32_t n_seqs, items, chunk;   // chunk: 128-key tiles per key range
  int32_t fin_rows;               // (candidate, head) rows of split sequences
  int64_t weight_rows;            // cached rows whose weight is updated (0: none)
  bool rab_per_head, vec, clear_err;
  bool out_f32;                   // out is float32 though q, k, v are bf16
  QcAttnSeq seqs[kQcMaxSeqs];
};
static_assert(sizeof(QcRowsParams) <= 4096 && sizeof(QcEvictParams) <= 4096 + 512 &&
                  sizeof(QcAttnParams) <= 8192,
              "kernel parameters");

constexpr int kQcKeyTile = 128;          // keys per tile (all kernels)
constexpr int kQcSimtQueries = 16;       // candidates per CTA of the CUDA-core kernel
constexpr int kQcFewQueries = 8;         // and of the one for few candidates

cudaError_t launch_qcache_append(const QcRowsParams &p, bool bf16, cudaStream_t st);
cudaError_t launch_qcache_read(const QcRowsParams &p, bool bf16, cudaStream_t st);
cudaError_t launch_qcache_evict(const QcEvictParams &p, int32_t max_len, int64_t move_blocks,
                                cudaStream_t st);
// Tensor cores: bf16, d_qk = d_v in {64, 128}; nq = 64 or 128 candidates per CTA.
cudaError_t launch_qcache_attn_tc(const QcAttnParams &p, int nq, cudaStream_t st);
// Warp-level products: the same types and sizes, 8 candidates per CTA.
cudaError_t launch_qcache_attn_few(const QcAttnParams &p, cudaStream_t st);
cudaError_t launch_qcache_attn_simt(const QcAttnParams &p, bool bf16, cudaStream_t st);
// Sums the partial outputs of split sequences and the weight partials
// (planes of `plane` candidates each).
cudaError_t launch_qcache_finish(const QcAttnParams &p, bool bf16, int plane, cudaStream_t st);

}  // namespace hstu
