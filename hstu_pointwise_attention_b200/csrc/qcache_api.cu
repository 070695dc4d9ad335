// qcache_api.cu -- entry points of the 4-bit history cache (include/hstu.h):
// argument checks, the per-launch sequence tables and key ranges, workspace
// layout and launches.  Host code only; nothing here allocates or waits.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <vector>

#include "../../include/hstu.h"
#include "api_common.h"
#include "qcache_host.h"

namespace hstu {
namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The cache's own fields.  `weight`: it has to hold weights.
hstu_status_t check_cache(const hstu_qcache_t *c, bool weight) {
  if (!c) return HSTU_ERR_INVALID_ARG;
  if (c->num_heads < 1 || c->num_heads > 4096) return HSTU_ERR_INVALID_ARG;
  for (int32_t d : {c->d_qk, c->d_v})
    if (d < 32 || d > 256 || d % 32) return HSTU_ERR_INVALID_ARG;
  if (c->rows < 0 || c->rows > (int64_t(1) << 40)) return HSTU_ERR_INVALID_ARG;
  if (c->rows == 0) return HSTU_OK;
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || !c->times || !c->pos ||
      (weight && !c->weight))
    return HSTU_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 16) ||
      !aligned(c->v_scales, 16) || !aligned(c->times, 8) || !aligned(c->pos, 4) ||
      !aligned(c->weight, 4))
    return HSTU_ERR_INVALID_ARG;
  return HSTU_OK;
}

QCacheView view_of(const hstu_qcache_t *c) {
  QCacheView v{};
  v.rows = c->rows;
  v.heads = c->num_heads;
  v.d_qk = c->d_qk;
  v.d_v = c->d_v;
  v.k_codes = static_cast<uint32_t *>(c->k_codes);
  v.v_codes = static_cast<uint32_t *>(c->v_codes);
  v.k_scales = c->k_scales;
  v.v_scales = c->v_scales;
  v.times = c->times;
  v.pos = c->pos;
  v.weight = c->weight;
  return v;
}

// [start, start + len) inside [0, rows).
bool in_rows(int64_t start, int64_t len, int64_t rows) {
  return start >= 0 && len >= 0 && len <= rows && start <= rows - len;
}

// No two regions [start[b], start[b] + len(b)) share a row.
template <class Len>
bool disjoint(const int64_t *start, Len len, int32_t B) {
  int64_t end = INT64_MIN;
  bool ascending = true;
  for (int32_t b = 0; b < B && ascending; ++b) {
    if (len(b) == 0) continue;
    ascending = start[b] >= end;
    end = start[b] + len(b);
  }
  if (ascending) return true;
  try {
    std::vector<std::pair<int64_t, int64_t>> r;
    r.reserve(size_t(B));
    for (int32_t b = 0; b < B; ++b)
      if (len(b) > 0) r.emplace_back(start[b], start[b] + len(b));
    std::sort(r.begin(), r.end());
    for (size_t i = 1; i < r.size(); ++i)
      if (r[i].first < r[i - 1].second) return false;
    return true;
  } catch (...) {   // no host memory for the sorted copy: compare all pairs
    for (int32_t a = 0; a < B; ++a)
      for (int32_t b = 0; b < a; ++b)
        if (len(a) > 0 && len(b) > 0 && start[a] < start[b] + len(b) &&
            start[b] < start[a] + len(a))
          return false;
    return true;
  }
}

bool overlap(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return std::max(x, y) < std::min(x + uintptr_t(a_bytes), y + uintptr_t(b_bytes));
}

// No buffer of one cache shares a byte with any buffer of the other.
bool apart(const hstu_qcache_t *x, const hstu_qcache_t *y) {
  struct Buf {
    const void *at;
    int64_t bytes;
  };
  auto bufs = [](const hstu_qcache_t *c, Buf (&b)[7]) {
    const int64_t R = c->rows, k = R * c->num_heads * c->d_qk, v = R * c->num_heads * c->d_v;
    const Buf all[7] = {{c->k_codes, k / 2},   {c->v_codes, v / 2}, {c->k_scales, k / 16},
                        {c->v_scales, v / 16}, {c->times, R * 8},   {c->pos, R * 4},
                        {c->weight, R * 4}};
    std::copy(all, all + 7, b);
  };
  Buf a[7], b[7];
  bufs(x, a);
  bufs(y, b);
  for (const Buf &i : a)
    for (const Buf &j : b)
      if (overlap(i.at, i.bytes, j.at, j.bytes)) return false;
  return true;
}

bool offsets_ok(const int64_t *off, int32_t B) {
  if (B > 0 && (!off || off[0] != 0)) return false;
  for (int32_t b = 0; b < B; ++b)
    if (off[b + 1] < off[b]) return false;
  return true;
}


// ---------------------------------------------------------------------------
// Append and read
// ---------------------------------------------------------------------------
template <class Tok, class Pos>
hstu_status_t run_rows(const hstu_qcache_t *cache, int32_t dtype, int32_t B, Tok tok,
                       const int64_t *rows, Pos pos, const void *k, int64_t k_rs, const void *v,
                       int64_t v_rs, const int64_t *ts, bool append, cudaStream_t st) {
  const int64_t per16 = dtype == HSTU_BF16 ? 8 : 4;
  QcRowsParams p{};
  p.cache = view_of(cache);
  p.k = k;
  p.v = v;
  p.k_rs = k_rs;
  p.v_rs = v_rs;
  p.ts = ts;
  p.k_magic = uint32_t((uint64_t(1) << 32) / uint32_t(cache->d_qk)) + 1;
  p.v_magic = uint32_t((uint64_t(1) << 32) / uint32_t(cache->d_v)) + 1;
  p.vec = aligned(k, 16) && aligned(v, 16) && k_rs % per16 == 0 && v_rs % per16 == 0;
  const int kw = cache->d_qk / 8, vw = cache->d_v / 8;   // units per head
  int64_t T = 0;
  for (int32_t b = 0; b < B; ++b) T += tok(b);
  p.lanes = std::min(T >= kQcManyRows ? 32 : 128, cache->num_heads * std::max(kw, vw));
  p.k_step = p.lanes % kw == 0 ? p.lanes / kw * cache->rows : 0;
  p.v_step = p.lanes % vw == 0 ? p.lanes / vw * cache->rows : 0;
  int64_t at = 0;
  for (int32_t b0 = 0; b0 < B; b0 += kQcMaxSeqs) {
    p.n_seqs = std::min(kQcMaxSeqs, B - b0);
    p.tok0 = at;
    for (int32_t i = 0; i < p.n_seqs; ++i) {
      p.seqs[i] = QcRows{at, rows[b0 + i], pos(b0 + i)};
      at += tok(b0 + i);
    }
    p.tok_end = at;
    if (p.tok_end == p.tok0) continue;
    const cudaError_t e = append ? launch_qcache_append(p, dtype == HSTU_BF16, st)
                                 : launch_qcache_read(p, dtype == HSTU_BF16, st);
    if (e != cudaSuccess) return HSTU_ERR_CUDA;
  }
  return HSTU_OK;
}

// ---------------------------------------------------------------------------
// Attention over the cache
// ---------------------------------------------------------------------------
struct AttnArgs {
  const hstu_attn_params_t *p;
  const hstu_qcache_t *cache;
  const int64_t *rows, *lens, *coff;
  const int32_t *pos;
  bool weight;
};

hstu_status_t check_attn(const AttnArgs &a, bool have_cache) {
  hstu_status_t st = validate_shape(a.p);
  if (st != HSTU_OK) return st;
  const hstu_attn_params_t &p = *a.p;
  if (p.batch < 0) return HSTU_ERR_INVALID_ARG;
  for (int32_t d : {p.d_qk, p.d_v})
    if (d < 32 || d % 32) return HSTU_ERR_INVALID_ARG;
  if (have_cache) {
    st = check_cache(a.cache, a.weight);
    if (st != HSTU_OK) return st;
    if (a.cache->num_heads != p.num_heads || a.cache->d_qk != p.d_qk || a.cache->d_v != p.d_v)
      return HSTU_ERR_INVALID_ARG;
    if (p.batch > 0 && (!a.rows || !a.pos)) return HSTU_ERR_INVALID_ARG;
  }
  if (p.batch > 0 && !a.lens) return HSTU_ERR_INVALID_ARG;
  if (!offsets_ok(a.coff, p.batch)) return HSTU_ERR_INVALID_ARG;
  int64_t all = 0;
  for (int32_t b = 0; b < p.batch; ++b) {
    const int64_t n = a.coff[b + 1] - a.coff[b], L = a.lens[b];
    if (L < 0 || n > p.max_seq_len || L > p.max_seq_len - n) return HSTU_ERR_INVALID_ARG;
    if (L > kQcMaxLen || n > kQcMaxLen) return HSTU_ERR_UNSUPPORTED;
    if (have_cache && !in_rows(a.rows[b], L, a.cache->rows)) return HSTU_ERR_INVALID_ARG;
    all += L;
  }
  // item and row counters of a launch are 32-bit
  const int64_t T = p.batch > 0 ? a.coff[p.batch] : 0;
  const int64_t most = int64_t(1) << 31;
  if (T >= most || T * p.num_heads >= most || all >= (int64_t(1) << 40))
    return HSTU_ERR_UNSUPPORTED;
  if (have_cache && a.weight &&
      !disjoint(a.rows, [&](int32_t b) { return a.lens[b]; }, p.batch))
    return HSTU_ERR_INVALID_ARG;
  return HSTU_OK;
}

// One launch's share of the call: sequences [b0, b0 + n_seqs), their key
// ranges and their places in the scratch buffers.
struct Share {
  bool tc, few;              // bf16 kernels: wide tiles; up to kQcFewQueries candidates each
  int nq, plane;             // candidates per CTA; candidates per weight partial
  int64_t acc_rows, wp;      // rows of `acc` (d_v floats each) and floats of `wpart` it uses
};

// How the keys are split.  A CTA holds `nq` candidates of one (sequence, head)
// and walks `chunk` 128-key tiles.  `slots` CTAs run at once.  A CTA's fixed
// cost (tables, queries, the output) is worth `fixed` tiles (the tcgen05 kernel's 9: of
// eleven shapes one depends on it, 4 x 1,024 on 8,192 with weights, 316 us up to 7
// tiles and 289 from 9 to 16), and a split adds
// the summing pass; the estimate below is the time in tiles: one chunk when all
// CTAs run at once, else the shared work plus half a CTA for the uneven end.
int32_t pick_chunk(const AttnArgs &a, int32_t b0, int32_t n_seqs, int nq, int64_t slots,
                   int64_t fixed) {
  const int64_t H = a.p->num_heads;
  uint32_t tiles[kQcMaxSeqs];        // sequences with candidates: 128-key tiles,
  int64_t ctas[kQcMaxSeqs];          // and CTAs per key range
  int32_t m = 0;
  int64_t most = 1, work = 0, all = 0;
  for (int32_t i = 0; i < n_seqs; ++i) {
    const int64_t n = a.coff[b0 + i + 1] - a.coff[b0 + i];
    if (n == 0) continue;
    const int64_t t = (a.lens[b0 + i] + kQcKeyTile - 1) / kQcKeyTile;
    tiles[m] = uint32_t(t > 1 ? t : 1);
    ctas[m] = H * ((n + nq - 1) / nq);
    most = std::max(most, t);
    work += ctas[m] * t;
    all += ctas[m];
    ++m;
  }
  auto count = [&](int64_t c) {
    const uint32_t d = uint32_t(c);
    int64_t items = 0;
    for (int32_t i = 0; i < m; ++i) items += ctas[i] * ((tiles[i] + d - 1) / d);
    return items;
  };
  int64_t best = most, best_cost = INT64_MAX;
  for (int waves = 0; waves <= 4; ++waves) {
    // the shortest chunk whose CTAs fit `waves` rounds; waves = 0: no split
    int64_t c = most;
    if (waves > 0) {
      // count(c) lies between work / c and work / c + all
      const int64_t room = slots * waves;
      int64_t lo = std::min(most, std::max<int64_t>(1, work / room)), hi = most;
      if (room > all) hi = std::max(lo, std::min(most, work / (room - all) + 1));
      while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (count(mid) <= room)
          hi = mid;
        else
          lo = mid + 1;
      }
      c = lo;
    }
    const int64_t items = count(c);
    int64_t cost = items <= slots ? 2 * slots * (c + fixed)
                                  : 2 * (work + items * fixed) + slots * (c + fixed);
    if (c < most) cost += 2 * slots * 2;
    if (cost < best_cost) {
      best_cost = cost;
      best = c;
    }
  }
  return int32_t(best);
}

// Fills the table of one launch.  acc_row, wp: first free places of the scratch.
void make_share(const AttnArgs &a, int32_t b0, int64_t acc_row, int64_t wp, QcAttnParams &p,
                Share &s) {
  const hstu_attn_params_t &ap = *a.p;
  const int64_t H = ap.num_heads;
  p.n_seqs = std::min(kQcMaxSeqs, ap.batch - b0);
  s.tc = ap.dtype == HSTU_BF16 && ap.impl == HSTU_IMPL_AUTO && ap.d_qk == ap.d_v &&
         (ap.d_qk == 64 || ap.d_qk == 128);
  if (s.tc) {
    // Warp-level products while no sequence has more than 8 candidates, else tcgen05
    // tiles of 64, or of 128 where some sequence has more.  Measured at 8 / 64
    // histories of 4,096 events (8 heads of 128), warp-level against 64-wide tiles: 8
    // candidates 21 / 104 us against 26 / 162, 9 (two of its tiles) 33 / 174
    // against 26 / 163.
    int64_t most = 0;
    for (int32_t b = b0; b < b0 + p.n_seqs; ++b) most = std::max(most, a.coff[b + 1] - a.coff[b]);
    s.few = most <= kQcFewQueries;
    s.nq = s.few ? kQcFewQueries : most <= 64 ? 64 : 128;
    s.plane = s.few ? kQcFewQueries : 64;
    p.chunk = s.few ? pick_chunk(a, b0, p.n_seqs, s.nq, 148 * 4, 1)
                    : pick_chunk(a, b0, p.n_seqs, s.nq, 148, 9);
  } else {
    s.few = false;
    s.nq = s.plane = kQcSimtQueries;
    p.chunk = pick_chunk(a, b0, p.n_seqs, s.nq, 148 * 4, 1);
  }
  s.acc_rows = s.wp = 0;
  int64_t items = 0, fin = 0, wrow = 0;
  for (int32_t i = 0; i < p.n_seqs; ++i) {
    const int32_t b = b0 + i;
    QcAttnSeq &q = p.seqs[i];
    q.row = a.rows ? a.rows[b] : 0;
    q.q0 = a.coff[b];
    q.len = int32_t(a.lens[b]);
    q.n = int32_t(a.coff[b + 1] - a.coff[b]);
    q.pos = a.pos ? a.pos[b] : 0;
    q.item0 = int32_t(items);
    q.fin0 = int32_t(fin);
    q.wrow0 = wrow;
    q.acc0 = acc_row + s.acc_rows;
    q.wp0 = wp + s.wp;
    const int32_t tiles = (q.len + kQcKeyTile - 1) / kQcKeyTile;
    q.splits = std::max(1, (tiles + p.chunk - 1) / p.chunk);
    items += int64_t((q.n + s.nq - 1) / s.nq) * q.splits;
    if (q.splits > 1) {
      fin += q.n * H;
      s.acc_rows += int64_t(q.splits) * q.n * H;
    }
    if (a.weight) {
      wrow += q.len;
      s.wp += int64_t((q.n + s.plane - 1) / s.plane) * H * q.len;
    }
  }
  p.items = int32_t(items);
  p.fin_rows = int32_t(fin);
  p.weight_rows = wrow;
}

// Workspace: error word, partial outputs, weight partials.
struct AttnWs {
  size_t acc, wpart, total;
};
AttnWs attn_layout(const AttnArgs &a) {
  AttnArgs shape = a;
  shape.rows = nullptr;
  shape.pos = nullptr;
  QcAttnParams p{};
  Share s{};
  int64_t rows = 0, wp = 0;
  for (int32_t b0 = 0; b0 < a.p->batch; b0 += kQcMaxSeqs) {
    make_share(shape, b0, rows, wp, p, s);
    rows += s.acc_rows;
    wp += s.wp;
  }
  AttnWs w{};
  w.acc = 256;
  w.wpart = align256(w.acc + size_t(rows) * a.p->d_v * sizeof(float));
  w.total = align256(w.wpart + size_t(wp) * sizeof(float));
  return w;
}

hstu_status_t run_attn(const AttnArgs &a, const int64_t *cand_ts, const void *q, const void *k,
                       const void *v, const float *rab_pos, const float *rab_time, float decay,
                       void *out, bool out_f32, const AttnWs &w, uint8_t *ws, bool clear_err,
                       cudaStream_t st) {
  const hstu_attn_params_t &ap = *a.p;
  const bool bf16 = ap.dtype == HSTU_BF16;
  const int64_t per16 = bf16 ? 8 : 4;
  QcAttnParams p{};
  p.cache = view_of(a.cache);
  p.q = q;
  p.k = k;
  p.v = v;
  p.out = out;
  p.q_rs = ap.q_row_stride;
  p.k_rs = ap.k_row_stride;
  p.v_rs = ap.v_row_stride;
  p.o_rs = ap.o_row_stride;
  p.cand_ts = cand_ts;
  p.rab_p = rab_pos;
  p.rab_t = rab_time;
  p.acc = reinterpret_cast<float *>(ws + w.acc);
  p.wpart = reinterpret_cast<float *>(ws + w.wpart);
  p.wait = WaitCtl{reinterpret_cast<uint32_t *>(ws), wait_limit_ns()};
  p.alpha = ap.alpha;
  p.scale = ap.silu_scale;
  p.decay = decay;
  p.nb_p = ap.num_pos_buckets;
  p.nb_t = ap.num_time_buckets;
  p.sub_bits = ap.time_bucket_sub_bits;
  p.rab_per_head = ap.rab_per_head != 0;
  p.vec = aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(out, 16) &&
          p.q_rs % per16 == 0 && p.k_rs % per16 == 0 && p.v_rs % per16 == 0 &&
          p.o_rs % per16 == 0;
  p.clear_err = clear_err;
  p.out_f32 = out_f32;
  int64_t rows = 0, wp = 0;
  Share s{};
  for (int32_t b0 = 0; b0 < ap.batch; b0 += kQcMaxSeqs) {
    make_share(a, b0, rows, wp, p, s);
    rows += s.acc_rows;
    wp += s.wp;
    if (p.items > 0) {
      const cudaError_t e = s.few  ? launch_qcache_attn_few(p, st)
                            : s.tc ? launch_qcache_attn_tc(p, s.nq, st)
                                 : launch_qcache_attn_simt(p, bf16, st);
      if (e != cudaSuccess) return HSTU_ERR_CUDA;
      p.clear_err = false;
    }
    if (launch_qcache_finish(p, bf16, s.plane, st) != cudaSuccess) return HSTU_ERR_CUDA;
  }
  if (p.clear_err && cudaMemsetAsync(ws, 0, 16, st) != cudaSuccess) return HSTU_ERR_CUDA;
  return HSTU_OK;
}

bool workspace_ok(const void *ws, size_t bytes, size_t need) {
  return ws && bytes >= need && aligned(ws, 256);
}

// ---------------------------------------------------------------------------
// Layer
// ---------------------------------------------------------------------------
// The attention's output A stays float32 up to the LayerNorm, which divides it by its
// deviation over the features: long histories average v, so A differs little between
// features (mean / deviation of 3 and more), and A in bf16 was most of y's error (of
// 2.8e-3 relative to 64 bits, with 2.0e-3 left; 8 x 256 candidates 96.4 us, so 98.2).
struct LayerQcWs {
  AttnWs attn;
  size_t proj, a, g, total;
};

hstu_status_t check_layer(const hstu_layer_params_t *lp, AttnArgs &a, hstu_attn_params_t &ap,
                          bool have_cache) {
  if (!lp) return HSTU_ERR_INVALID_ARG;
  if (lp->d_model < 8 || lp->d_model > 8192 || (lp->d_model & 7)) return HSTU_ERR_INVALID_ARG;
  if (!(lp->ln_eps > 0.f) || !std::isfinite(lp->ln_eps)) return HSTU_ERR_INVALID_ARG;
  ap = lp->attn;
  const int64_t H = ap.num_heads, F = H * ap.d_v, n1 = 2 * (F + H * ap.d_qk);
  ap.q_row_stride = ap.k_row_stride = ap.v_row_stride = n1;
  ap.o_row_stride = F;
  a.p = &ap;
  hstu_status_t st = check_attn(a, have_cache);
  if (st != HSTU_OK) return st;
  if (ap.dtype != HSTU_BF16) return HSTU_ERR_UNSUPPORTED;
  // the row lengths the LayerNorm gating kernel is built for
  if (F != 32 && F != 64 && F != 128 && F != 256 && F != 512 && F != 1024)
    return HSTU_ERR_UNSUPPORTED;
  return HSTU_OK;
}

LayerQcWs layer_layout(const AttnArgs &a) {
  LayerQcWs w{};
  const hstu_attn_params_t &ap = *a.p;
  const int64_t T = ap.batch > 0 ? a.coff[ap.batch] : 0, H = ap.num_heads, F = H * ap.d_v;
  w.attn = attn_layout(a);   // its error word (offset 0) serves the whole layer
  w.proj = align256(w.attn.total);
  w.a = align256(w.proj + size_t(T) * 2 * (F + H * ap.d_qk) * 2);
  w.g = align256(w.a + size_t(T) * F * 4);
  w.total = align256(w.g + size_t(T) * F * 2);
  return w;
}

}  // namespace
}  // namespace hstu

using namespace hstu;

extern "C" {

hstu_status_t hstu_qcache_append(const hstu_qcache_t *cache, int32_t dtype, int32_t batch,
                                 const int64_t *tok_offsets_host, const int64_t *rows_host,
                                 const int32_t *pos_host, const void *k, int64_t k_row_stride,
                                 const void *v, int64_t v_row_stride,
                                 const int64_t *timestamps_dev, void *stream) {
  hstu_status_t st = check_cache(cache, false);
  if (st != HSTU_OK) return st;
  if (dtype != HSTU_F32 && dtype != HSTU_BF16) return HSTU_ERR_INVALID_ARG;
  if (batch < 0 || !offsets_ok(tok_offsets_host, batch)) return HSTU_ERR_INVALID_ARG;
  if (batch > 0 && (!rows_host || !pos_host)) return HSTU_ERR_INVALID_ARG;
  const int64_t T = batch > 0 ? tok_offsets_host[batch] : 0;
  if (T >= (int64_t(1) << 31)) return HSTU_ERR_UNSUPPORTED;
  auto len = [&](int32_t b) { return tok_offsets_host[b + 1] - tok_offsets_host[b]; };
  for (int32_t b = 0; b < batch; ++b) {
    if (!in_rows(rows_host[b], len(b), cache->rows)) return HSTU_ERR_INVALID_ARG;
    if (len(b) > 0 && int64_t(pos_host[b]) + len(b) - 1 > INT32_MAX) return HSTU_ERR_INVALID_ARG;
  }
  if (!disjoint(rows_host, len, batch)) return HSTU_ERR_INVALID_ARG;
  if (k_row_stride < int64_t(cache->num_heads) * cache->d_qk ||
      v_row_stride < int64_t(cache->num_heads) * cache->d_v)
    return HSTU_ERR_INVALID_ARG;
  if (T == 0) return HSTU_OK;
  const uintptr_t es = dtype == HSTU_BF16 ? 2 : 4;
  if (!k || !v || !timestamps_dev || !aligned(k, es) || !aligned(v, es) ||
      !aligned(timestamps_dev, 8))
    return HSTU_ERR_INVALID_ARG;
  return run_rows(cache, dtype, batch, len, rows_host,
                  [&](int32_t b) { return int64_t(pos_host[b]); }, k, k_row_stride, v,
                  v_row_stride, timestamps_dev, true, static_cast<cudaStream_t>(stream));
}

hstu_status_t hstu_qcache_read(const hstu_qcache_t *cache, int32_t dtype, int32_t batch,
                               const int64_t *rows_host, const int64_t *lens_host, void *k,
                               int64_t k_row_stride, void *v, int64_t v_row_stride,
                               void *stream) {
  hstu_status_t st = check_cache(cache, false);
  if (st != HSTU_OK) return st;
  if (dtype != HSTU_F32 && dtype != HSTU_BF16) return HSTU_ERR_INVALID_ARG;
  if (batch < 0 || (batch > 0 && (!rows_host || !lens_host))) return HSTU_ERR_INVALID_ARG;
  int64_t T = 0;
  for (int32_t b = 0; b < batch; ++b) {
    if (!in_rows(rows_host[b], lens_host[b], cache->rows)) return HSTU_ERR_INVALID_ARG;
    T += lens_host[b];
    if (T >= (int64_t(1) << 31)) return HSTU_ERR_UNSUPPORTED;
  }
  if (k_row_stride < int64_t(cache->num_heads) * cache->d_qk ||
      v_row_stride < int64_t(cache->num_heads) * cache->d_v)
    return HSTU_ERR_INVALID_ARG;
  if (T == 0) return HSTU_OK;
  const uintptr_t es = dtype == HSTU_BF16 ? 2 : 4;
  if (!k || !v || !aligned(k, es) || !aligned(v, es)) return HSTU_ERR_INVALID_ARG;
  return run_rows(cache, dtype, batch, [&](int32_t b) { return lens_host[b]; }, rows_host,
                  [](int32_t) { return int64_t(0); }, k, k_row_stride, v, v_row_stride, nullptr,
                  false, static_cast<cudaStream_t>(stream));
}

static hstu_status_t evict_sizes(int32_t batch, const int64_t *lens, const int64_t *budgets,
                                 int64_t *kept) {
  if (batch < 0 || (batch > 0 && (!lens || !budgets))) return HSTU_ERR_INVALID_ARG;
  *kept = 0;
  for (int32_t b = 0; b < batch; ++b) {
    if (lens[b] < 0 || budgets[b] < 0) return HSTU_ERR_INVALID_ARG;
    if (lens[b] > kQcMaxLen) return HSTU_ERR_UNSUPPORTED;
    *kept += std::min(lens[b], budgets[b]);
  }
  return *kept < (int64_t(1) << 36) ? HSTU_OK : HSTU_ERR_UNSUPPORTED;
}

hstu_status_t hstu_qcache_evict_workspace_size(int32_t batch, const int64_t *lens_host,
                                               const int64_t *budgets_host, size_t *bytes) {
  if (!bytes) return HSTU_ERR_INVALID_ARG;
  int64_t kept;
  hstu_status_t st = evict_sizes(batch, lens_host, budgets_host, &kept);
  if (st != HSTU_OK) return st;
  *bytes = 2 * align256(size_t(kept) * sizeof(int32_t));
  return HSTU_OK;
}

hstu_status_t hstu_qcache_evict(const hstu_qcache_t *src, const hstu_qcache_t *dst,
                                int32_t batch, const int64_t *rows_host,
                                const int64_t *lens_host, const int64_t *budgets_host,
                                const int32_t *keep_pos_host, const int64_t *dst_rows_host,
                                void *workspace, size_t workspace_bytes, void *stream) {
  hstu_status_t st = check_cache(src, true);
  if (st == HSTU_OK) st = check_cache(dst, true);
  if (st != HSTU_OK) return st;
  if (src->num_heads != dst->num_heads || src->d_qk != dst->d_qk || src->d_v != dst->d_v)
    return HSTU_ERR_INVALID_ARG;
  int64_t kept;
  st = evict_sizes(batch, lens_host, budgets_host, &kept);
  if (st != HSTU_OK) return st;
  if (batch > 0 && (!rows_host || !dst_rows_host || !keep_pos_host)) return HSTU_ERR_INVALID_ARG;
  auto keep = [&](int32_t b) { return std::min(lens_host[b], budgets_host[b]); };
  bool in_place = src->rows == dst->rows && src->k_codes == dst->k_codes &&
                  src->v_codes == dst->v_codes && src->k_scales == dst->k_scales &&
                  src->v_scales == dst->v_scales && src->times == dst->times &&
                  src->pos == dst->pos && src->weight == dst->weight;
  for (int32_t b = 0; b < batch; ++b) {
    if (!in_rows(rows_host[b], lens_host[b], src->rows) ||
        !in_rows(dst_rows_host[b], keep(b), dst->rows))
      return HSTU_ERR_INVALID_ARG;
    // within one cache rows only move inside their own region
    if (in_place && dst_rows_host[b] != rows_host[b]) return HSTU_ERR_INVALID_ARG;
  }
  if (in_place) {
    if (!disjoint(rows_host, [&](int32_t b) { return lens_host[b]; }, batch))
      return HSTU_ERR_INVALID_ARG;
  } else {
    if (!disjoint(dst_rows_host, keep, batch)) return HSTU_ERR_INVALID_ARG;
    if (!apart(src, dst)) return HSTU_ERR_INVALID_ARG;
  }
  if (kept == 0) return HSTU_OK;
  const size_t half = align256(size_t(kept) * sizeof(int32_t));
  if (!workspace_ok(workspace, workspace_bytes, 2 * half)) return HSTU_ERR_WORKSPACE;
  QcEvictParams p{};
  p.src = view_of(src);
  p.dst = view_of(dst);
  p.map = static_cast<int32_t *>(workspace);
  p.movers = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + half);
  p.in_place = in_place;
  // 32 rows per block, 8 while that leaves SMs without one
  p.move_rows = kept >= 32 * 4 * 148 ? 32 : 8;
  int64_t map0 = 0;
  for (int32_t b0 = 0; b0 < batch; b0 += kQcMaxSeqs) {
    p.n_seqs = std::min(kQcMaxSeqs, batch - b0);
    int64_t blocks = 0;
    int32_t longest = 1;
    for (int32_t i = 0; i < p.n_seqs; ++i) {
      const int32_t b = b0 + i;
      QcEvictSeq &s = p.seqs[i];
      s.row = rows_host[b];
      s.dst_row = dst_rows_host[b];
      s.map0 = map0;
      s.block0 = blocks;
      s.len = int32_t(lens_host[b]);
      s.keep = int32_t(keep(b));
      s.keep_pos = keep_pos_host[b];
      // nothing to move: everything is kept where it is
      if (in_place && s.keep == s.len) s.keep = s.len = 0;
      map0 += keep(b);
      blocks += (s.keep + p.move_rows - 1) / p.move_rows;
      longest = std::max(longest, s.len);
    }
    if (blocks == 0) continue;
    if (blocks >= (int64_t(1) << 31)) return HSTU_ERR_UNSUPPORTED;
    if (launch_qcache_evict(p, longest, blocks, static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return HSTU_ERR_CUDA;
  }
  return HSTU_OK;
}

hstu_status_t hstu_attn_candidates_qcache_workspace_size(const hstu_attn_params_t *params,
                                                         const int64_t *cache_lens_host,
                                                         const int64_t *cand_offsets_host,
                                                         int32_t update_weight, size_t *bytes) {
  if (!bytes) return HSTU_ERR_INVALID_ARG;
  AttnArgs a{params, nullptr, nullptr, cache_lens_host, cand_offsets_host, nullptr,
             update_weight != 0};
  hstu_status_t st = check_attn(a, false);
  if (st != HSTU_OK) return st;
  *bytes = attn_layout(a).total;
  return HSTU_OK;
}

hstu_status_t hstu_attn_fwd_candidates_qcache(
    const hstu_attn_params_t *params, const hstu_qcache_t *cache, const int64_t *cache_rows_host,
    const int64_t *cache_lens_host, const int64_t *cand_offsets_host,
    const int32_t *cand_pos_host, const int64_t *cand_timestamps_dev, const void *q,
    const void *k, const void *v, const float *rab_pos, const float *rab_time,
    int32_t update_weight, float weight_decay, void *out, void *workspace,
    size_t workspace_bytes, void *stream) {
  AttnArgs a{params, cache, cache_rows_host, cache_lens_host, cand_offsets_host, cand_pos_host,
             update_weight != 0};
  hstu_status_t st = check_attn(a, true);
  if (st != HSTU_OK) return st;
  if (a.weight && !std::isfinite(weight_decay)) return HSTU_ERR_INVALID_ARG;
  const int64_t T = params->batch > 0 ? cand_offsets_host[params->batch] : 0;
  const uintptr_t es = params->dtype == HSTU_BF16 ? 2 : 4;
  if (T > 0 && (!cand_timestamps_dev || !q || !k || !v || !rab_pos || !rab_time || !out ||
                !aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(out, es) ||
                !aligned(cand_timestamps_dev, 8) || !aligned(rab_pos, 4) || !aligned(rab_time, 4)))
    return HSTU_ERR_INVALID_ARG;
  const AttnWs w = attn_layout(a);
  if (!workspace_ok(workspace, workspace_bytes, w.total)) return HSTU_ERR_WORKSPACE;
  return run_attn(a, cand_timestamps_dev, q, k, v, rab_pos, rab_time, weight_decay, out,
                  false, w, static_cast<uint8_t *>(workspace), true,
                  static_cast<cudaStream_t>(stream));
}

hstu_status_t hstu_layer_candidates_qcache_workspace_size(const hstu_layer_params_t *params,
                                                          const int64_t *cache_lens_host,
                                                          const int64_t *cand_offsets_host,
                                                          int32_t update_weight, size_t *bytes) {
  if (!bytes) return HSTU_ERR_INVALID_ARG;
  AttnArgs a{nullptr, nullptr, nullptr, cache_lens_host, cand_offsets_host, nullptr,
             update_weight != 0};
  hstu_attn_params_t ap;
  hstu_status_t st = check_layer(params, a, ap, false);
  if (st != HSTU_OK) return st;
  *bytes = layer_layout(a).total;
  return HSTU_OK;
}

hstu_status_t hstu_layer_fwd_candidates_qcache(
    const hstu_layer_params_t *params, const hstu_qcache_t *cache,
    const int64_t *cache_rows_host, const int64_t *cache_lens_host,
    const int64_t *cand_offsets_host, const int32_t *cand_pos_host,
    const int64_t *cand_timestamps_dev, const void *x_cand, const void *w1, const float *b1,
    const float *ln_gamma, const float *ln_beta, const void *w2, const float *b2,
    const float *rab_pos, const float *rab_time, int32_t update_weight, float weight_decay,
    void *y_cand, void *proj_out, void *workspace, size_t workspace_bytes, void *stream) {
  AttnArgs a{nullptr, cache, cache_rows_host, cache_lens_host, cand_offsets_host, cand_pos_host,
             update_weight != 0};
  hstu_attn_params_t ap;
  hstu_status_t st = check_layer(params, a, ap, true);
  if (st != HSTU_OK) return st;
  if (a.weight && !std::isfinite(weight_decay)) return HSTU_ERR_INVALID_ARG;
  const int64_t T = ap.batch > 0 ? cand_offsets_host[ap.batch] : 0;
  if (T > 0 && (!cand_timestamps_dev || !x_cand || !w1 || !b1 || !ln_gamma || !ln_beta || !w2 ||
                !b2 || !rab_pos || !rab_time || !y_cand))
    return HSTU_ERR_INVALID_ARG;
  if (!aligned(cand_timestamps_dev, 8) || !aligned(x_cand, 2) || !aligned(w1, 2) ||
      !aligned(w2, 2) || !aligned(y_cand, 2) || !aligned(b1, 4) || !aligned(ln_gamma, 4) ||
      !aligned(ln_beta, 4) || !aligned(b2, 4) || !aligned(rab_pos, 4) || !aligned(rab_time, 4))
    return HSTU_ERR_INVALID_ARG;
  if (proj_out && !aligned(proj_out, 16)) return HSTU_ERR_INVALID_ARG;
  // x is read again behind the first rows of y, and the projection behind both
  const int64_t x_bytes = T * params->d_model * 2,
                p_bytes = T * 4 * ap.num_heads * (ap.d_v + ap.d_qk);
  if (overlap(x_cand, x_bytes, y_cand, x_bytes) ||
      (proj_out && (overlap(proj_out, p_bytes, x_cand, x_bytes) ||
                    overlap(proj_out, p_bytes, y_cand, x_bytes))))
    return HSTU_ERR_INVALID_ARG;
  const LayerQcWs lw = layer_layout(a);
  if (!workspace_ok(workspace, workspace_bytes, lw.total)) return HSTU_ERR_WORKSPACE;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  uint32_t *err = reinterpret_cast<uint32_t *>(ws);
  if (cudaMemsetAsync(err, 0, 16, cs) != cudaSuccess) return HSTU_ERR_CUDA;
  if (T == 0)   // no candidate rows; the weights still decay
    return run_attn(a, nullptr, nullptr, nullptr, nullptr, rab_pos, rab_time, weight_decay,
                    nullptr, true, lw.attn, ws, false, cs);
  const int64_t H = ap.num_heads, dqk = ap.d_qk, D = params->d_model, F = H * ap.d_v,
                n1 = 2 * (F + H * dqk);
  uint8_t *proj = proj_out ? static_cast<uint8_t *>(proj_out) : ws + lw.proj;
  uint8_t *att = ws + lw.a, *g = ws + lw.g;
  const WaitCtl wc{err, wait_limit_ns()};
  cudaError_t e = launch_gemm(x_cand, D, w1, D, b1, nullptr, 0, proj, n1, T, n1, D, kEpiBiasSilu,
                              wc, cs);
  if (e != cudaSuccess) return HSTU_ERR_CUDA;
  st = run_attn(a, cand_timestamps_dev, proj + 2 * (2 * F), proj + 2 * (2 * F + H * dqk),
                proj + 2 * F, rab_pos, rab_time, weight_decay, att, true, lw.attn, ws, false, cs);
  if (st != HSTU_OK) return st;
  e = launch_ln_gate_f32(reinterpret_cast<const float *>(att), F, proj, n1, ln_gamma, ln_beta,
                         params->ln_eps, g, F, T, int32_t(F), cs);
  if (e != cudaSuccess) return HSTU_ERR_CUDA;
  e = launch_gemm(g, F, w2, F, b2, params->residual ? x_cand : nullptr, D, y_cand, D, T, D, F,
                  params->residual ? kEpiBiasResidual : kEpiBias, wc, cs);
  return e == cudaSuccess ? HSTU_OK : HSTU_ERR_CUDA;
}

}  // extern "C"
