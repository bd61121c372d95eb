// C ABI of the rotary operator and the 8-bit cache: argument checks, workspace
// layout, launches.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "../../include/specverify.h"
#include "common.cuh"
#include "internal.h"
#include "qcache.h"

namespace sv {

namespace {

constexpr int kDefaultSplit = 1024;
constexpr int kMaxSplitTokens = 4096;
constexpr int kSplitGrain = 128;
constexpr int kMaxQSplits = 8192;        // splits of one sequence
constexpr int kMaxPagesPerSeq = 1 << 24; // positions stay below 2^30
constexpr int kMaxOffset = 65536;
constexpr int kMaxGridY = 65535;
constexpr int64_t kMaxRowStride = 1 << 26;   // elements: 32 rows on stay within 32 bits

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
inline int status_of(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA; }
inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Checks a configuration and forms its frequencies (f may be null).
int rope_frequencies(const spec_rope_config* r, int head_dim, double* f) {
  if (!r || head_dim < 2 || head_dim > SPEC_ROPE_MAX_DIM) return SPEC_EINVAL;
  if (r->layout != SPEC_ROPE_HALF && r->layout != SPEC_ROPE_INTERLEAVED) return SPEC_EINVAL;
  if (r->span < 2 || r->span % 2 || r->span > head_dim || r->n_rot < 0 || r->n_rot > r->span / 2)
    return SPEC_EINVAL;
  if (r->scaling < SPEC_ROPE_PLAIN || r->scaling > SPEC_ROPE_PARTS) return SPEC_EINVAL;
  // (the kernels take the magnitude in binary32)
  if (!(r->theta > 0.0) || !isfinite(r->theta) || !(r->magnitude >= FLT_MIN) || r->magnitude > FLT_MAX)
    return SPEC_EINVAL;
  if (r->scaling != SPEC_ROPE_PLAIN && (!(r->factor >= 1.0) || !isfinite(r->factor))) return SPEC_EINVAL;
  if (r->scaling == SPEC_ROPE_RAISED && r->span < 4) return SPEC_EINVAL;
  if (r->scaling == SPEC_ROPE_PARTS &&
      (!(r->original > 0.0) || !isfinite(r->original) || !(r->turns_lo >= 0.0) ||
       !(r->turns_hi > r->turns_lo) || !isfinite(r->turns_hi)))
    return SPEC_EINVAL;
  double base = r->theta;
  if (r->scaling == SPEC_ROPE_RAISED) base *= pow(r->factor, (double)r->span / (r->span - 2));
  if (!isfinite(base)) return SPEC_EINVAL;
  // base^(-2j / span) as a product of two powers (16 + 8 of them instead of 128, of
  // 50 ns each, in every call): off by 3 x 2^-53 at most
  double fine[8], coarse = 1.0;
  for (int j = 0; j < 8 && j < r->n_rot; ++j) fine[j] = pow(base, -2.0 * j / r->span);
  for (int j = 0; j < r->n_rot; ++j) {
    if (j > 0 && j % 8 == 0) coarse = pow(base, -2.0 * j / r->span);
    double g = coarse * fine[j % 8];
    if (r->scaling == SPEC_ROPE_LINEAR) g /= r->factor;
    if (r->scaling == SPEC_ROPE_PARTS) {
      double w = (r->original * g / (2.0 * M_PI) - r->turns_lo) / (r->turns_hi - r->turns_lo);
      w = w < 0.0 ? 0.0 : (w > 1.0 ? 1.0 : w);
      g = (1.0 - w) * g / r->factor + w * g;
    }
    if (!isfinite(g)) return SPEC_EINVAL;
    if (f) f[j] = g;
  }
  return SPEC_OK;
}

// Kernel arguments of a configuration; none (r null) turns nothing.
int rope_args(const spec_rope_config* r, int head_dim, RopeArgs* a) {
  *a = RopeArgs{};
  a->span = 2;
  a->magnitude = 1.0;
  if (!r) return SPEC_OK;
  double f[kMaxPairs];
  const int rc = rope_frequencies(r, head_dim, f);
  if (rc) return rc;
  a->layout = r->layout;
  a->span = r->span;
  a->n_rot = r->n_rot;
  a->magnitude = r->magnitude;
  for (int j = 0; j < r->n_rot; ++j) {
    const double turns = f[j] / (2.0 * M_PI);
    a->step[j] = static_cast<uint64_t>((turns - floor(turns)) * 0x1p64);   // below 2^64: the fraction is below 1
  }
  return SPEC_OK;
}

int check_cache(const spec_qcache* c) {
  if (!c || !c->k_pool || !c->v_pool || !c->k_scale || !c->v_scale) return SPEC_EINVAL;
  if (c->n_kv_heads < 1 || c->num_pages < 1) return SPEC_EINVAL;
  if (c->page_size != SPEC_PAGE_SIZE) return SPEC_EUNSUPPORTED;
  if (c->head_dim != 128 && c->head_dim != 256) return SPEC_EUNSUPPORTED;
  if (c->block_tokens != 16 && c->block_tokens != 32 && c->block_tokens != 64) return SPEC_EUNSUPPORTED;
  if (c->split_tokens < 0 || c->split_tokens % kSplitGrain || c->split_tokens > kMaxSplitTokens)
    return SPEC_EINVAL;
  if (!aligned(c->k_pool, 16) || !aligned(c->v_pool, 16) || !aligned(c->k_scale, 16) ||
      !aligned(c->v_scale, 16))
    return SPEC_EINVAL;
  if (c->n_kv_heads > kMaxGridY) return SPEC_EUNSUPPORTED;
  if ((uint64_t)c->num_pages * c->n_kv_heads * c->page_size > 0x7fffffffull) return SPEC_EUNSUPPORTED;
  return SPEC_OK;
}

int split_of(const spec_qcache* c) { return c->split_tokens > 0 ? c->split_tokens : kDefaultSplit; }

struct AttnLayout {
  size_t codes, scale, part_o, part_ml, total;
  int split, n_splits;
};

// Split of a call's attention.  Verify and decode calls (n <= SPEC_MAX_K + 1) take
// the cache's, so that a row's result depends on neither n nor the batch.  A
// prompt chunk has row blocks enough to fill the GPU, and a split's partial
// results and its join cost it more than they give (256 rows over 8k of context,
// 32 / 4 heads, by 64 rows: 296 us in three splits, 230 in one, which needs no join): it takes
// the number of splits of the least cost below, up to four items an SM and the
// kernel's limit of 256 scales an item.
constexpr int kItemsWanted = 4 * 148;
int call_split(const spec_qcache* c, int n_q_heads, int64_t B, int n, int max_pages) {
  const int split = split_of(c);
  if (n <= SPEC_MAX_K + 1) return split;
  const int cap = 256 * c->block_tokens;
  const int64_t rows = (int64_t)(n_q_heads / c->n_kv_heads) * n;
  const int rp = qattn_rows(n, rows);
  const int64_t groups = B * c->n_kv_heads * ((rows + rp - 1) / rp);
  const int64_t most = (kItemsWanted + groups - 1) / groups, T = (int64_t)max_pages * SPEC_PAGE_SIZE;
  int64_t best = 0, least = INT64_MAX;
  for (int64_t w = 1; w <= most; ++w) {
    int64_t e = ((T + w - 1) / w + kSplitGrain - 1) / kSplitGrain * kSplitGrain;
    if (e < split) e = split;
    if (e > cap) e = cap;
    // key blocks of the busiest SM, two more an item, and the join: 1/40 block an item
    const int64_t parts = (T + e - 1) / e;
    const int64_t cost = (groups * parts + 147) / 148 * (e / kQBlk + 2) + (parts > 1 ? groups * parts / 40 : 0);
    if (cost < least) {
      least = cost;
      best = e;
    }
    if (e == split) break;
  }
  return (int)best;
}

// False where the counts are out of range.
bool attn_layout(const spec_qcache* c, int n_q_heads, int B, int n, int max_pages, int window,
                 AttnLayout* s) {
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads || B < 1 || n < 1 || n > SPEC_MAX_PREFILL ||
      max_pages < 1 || max_pages > kMaxPagesPerSeq || window < 0)
    return false;
  s->split = call_split(c, n_q_heads, B, n, max_pages);
  const int64_t splits = ((int64_t)max_pages * SPEC_PAGE_SIZE + s->split - 1) / s->split;
  if (window == 0 && splits > kMaxQSplits) return false;
  s->n_splits = qcache_splits(max_pages, n, window, s->split);
  if (s->n_splits > kMaxQSplits) return false;
  const uint64_t rows = (uint64_t)B * n * n_q_heads;     // (sequence, KV head, row)
  if (rows > 0x3fffffffull) return false;
  // what the kernels count and divide in 32 bits: rows of a KV head by its query
  // heads, and twice the key blocks and items of all (sequence, KV head, row block)
  const uint64_t G = n_q_heads / c->n_kv_heads, per_head = n * G;
  if (per_head * G > 0xffffffffull ||
      (uint64_t)B * c->n_kv_heads * ((per_head + 31) / 32) * ((uint64_t)max_pages + 2) > 0x3fffffffull)
    return false;
  const uint64_t slots = rows * s->n_splits, D = c->head_dim;
  size_t off = kWsHeaderBytes;
  s->codes = off;   off = up256(off + 2 * rows * D);
  s->scale = off;   off = up256(off + rows * 4);
  s->part_o = off;  off = up256(off + slots * D * 4);
  s->part_ml = off; off = up256(off + slots * 8);
  s->total = off;
  return true;
}

// Bytes for any call up to these sizes.  A call of fewer sequences or rows may
// take a shorter split: with n <= SPEC_MAX_K + 1 the cache's own (of which it may have
// kMaxQSplits, so a chunk's table may be wider than such a call's), beyond that one
// that leaves at most kItemsWanted + (row blocks) items of 64 rows.
size_t attn_bytes(const spec_qcache* c, int n_q_heads, int B, int n, int max_pages, int window) {
  AttnLayout s;
  if (!attn_layout(c, n_q_heads, B, n, max_pages, window, &s)) return 0;
  size_t total = s.total;
  if (n > SPEC_MAX_K + 1) {
    AttnLayout v;
    const int64_t widest = (int64_t)kMaxQSplits * split_of(c) / SPEC_PAGE_SIZE;
    if (!attn_layout(c, n_q_heads, B, SPEC_MAX_K + 1, (int)(max_pages < widest ? max_pages : widest), window, &v)) return 0;
    const uint64_t rows = (uint64_t)B * n * n_q_heads, blocks = rows / 64 + (uint64_t)B * c->n_kv_heads;
    const uint64_t cap = ((uint64_t)max_pages * SPEC_PAGE_SIZE + 4095) / 4096;
    const uint64_t slots = 128 * (kItemsWanted + 2 * blocks) + rows * (cap + 1);
    const size_t most = s.part_o + slots * ((size_t)c->head_dim * 4 + 8) + 512;
    total = most > v.total ? most : v.total;
  }
  return total;
}

QCacheArgs cache_args(const spec_qcache* c, const int32_t* table, int max_pages, const int32_t* lens,
                      void* ws) {
  QCacheArgs a{};
  a.dim = c->head_dim;
  a.n_kv_heads = c->n_kv_heads;
  a.num_pages = c->num_pages;
  a.max_pages = max_pages;
  a.block = c->block_tokens;
  a.k = static_cast<uint8_t*>(c->k_pool);
  a.v = static_cast<uint8_t*>(c->v_pool);
  a.ks = static_cast<float*>(c->k_scale);
  a.vs = static_cast<float*>(c->v_scale);
  a.block_table = table;
  a.seq_lens = lens;
  a.status = ws_header(ws).status;
  return a;
}

int check_write(const spec_qcache* c, const int32_t* table, int max_pages, const int32_t* lens, int B,
                int n, const void* k_new, int64_t k_row, const void* v_new, int64_t v_row) {
  if (!table || !lens || !k_new || !v_new) return SPEC_EINVAL;
  if (B < 1 || n < 0 || n > SPEC_QCACHE_MAX_WRITE || max_pages < 1 || max_pages > kMaxPagesPerSeq)
    return SPEC_EINVAL;
  if (B > kMaxGridY / 2) return SPEC_EUNSUPPORTED;
  const int64_t width = (int64_t)c->n_kv_heads * c->head_dim;
  if (k_row > kMaxRowStride || v_row > kMaxRowStride) return SPEC_EUNSUPPORTED;
  if (k_row < width || v_row < width || k_row % 8 || v_row % 8 || !aligned(k_new, 16) || !aligned(v_new, 16))
    return SPEC_EINVAL;
  return SPEC_OK;
}

int run_write(const spec_qcache* c, const RopeArgs& r, const int32_t* table, int max_pages,
              const int32_t* lens, int B, int n, const void* k_new, int64_t k_row, const void* v_new,
              int64_t v_row, void* ws, cudaStream_t st) {
  QWriteArgs a{};
  a.c = cache_args(c, table, max_pages, lens, ws);
  a.B = B;
  a.n = n;
  a.k_new = static_cast<const uint16_t*>(k_new);
  a.v_new = static_cast<const uint16_t*>(v_new);
  a.k_row = k_row;
  a.v_row = v_row;
  return status_of(launch_qcache_write(r, a, st));
}

struct AttnCall {
  const void* q;
  int64_t q_row;
  int n_q_heads;
  const int32_t* table;
  int max_pages;
  const int32_t* lens;
  int B, n, q_offset, kv_extra, window;
  float scale;
  void* out;
  void* ws;
  size_t ws_bytes;
};

int check_attn(const spec_qcache* c, const AttnCall& a, AttnLayout* s) {
  if (!a.q || !a.table || !a.lens || !a.out || !a.ws) return SPEC_EINVAL;
  if (a.q_offset < 0 || a.q_offset > kMaxOffset || a.kv_extra < 0 || a.kv_extra > kMaxOffset)
    return SPEC_EINVAL;
  if (!isfinite(a.scale) || a.scale < 0.f) return SPEC_EINVAL;
  if (a.B < 1 || a.n < 1 || a.n > SPEC_MAX_PREFILL || a.n_q_heads < 1 || a.n_q_heads % c->n_kv_heads ||
      a.max_pages < 1 || a.window < 0)
    return SPEC_EINVAL;
  if (a.B > kMaxGridY) return SPEC_EUNSUPPORTED;
  const int64_t width = (int64_t)a.n_q_heads * c->head_dim;
  if (a.q_row < width || a.q_row % 8 || !aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.ws, 256))
    return SPEC_EINVAL;
  if (!attn_layout(c, a.n_q_heads, a.B, a.n, a.max_pages, a.window, s)) return SPEC_EUNSUPPORTED;
  return a.ws_bytes < s->total ? SPEC_EINVAL : SPEC_OK;
}

int run_attn(const spec_qcache* c, const RopeArgs& r, const AttnCall& k, const AttnLayout& s,
             cudaStream_t st) {
  uint8_t* ws = static_cast<uint8_t*>(k.ws);
  QAttnArgs a{};
  a.c = cache_args(c, k.table, k.max_pages, k.lens, k.ws);
  a.B = k.B;
  a.n = k.n;
  a.G = k.n_q_heads / c->n_kv_heads;
  a.rows = k.n * a.G;
  a.q_offset = k.q_offset;
  a.kv_extra = k.kv_extra;
  a.window = k.window;
  a.split = s.split;
  a.by_split = make_div(s.split / kQBlk);   // up to 2^7 of at most 2^23 blocks
  a.by_cost = make_div(s.split / kQBlk + 1);
  a.by_G = make_div(a.G);
  a.n_splits = s.n_splits;
  a.q = static_cast<const uint16_t*>(k.q);
  a.q_row = k.q_row;
  const double scale = k.scale > 0.f ? (double)k.scale : 1.0 / sqrt((double)c->head_dim);
  a.scale_log2 = (float)(scale * 1.4426950408889634);
  a.q_codes = ws + s.codes;
  a.q_scale = reinterpret_cast<float*>(ws + s.scale);
  a.part_o = reinterpret_cast<float*>(ws + s.part_o);
  a.part_ml = reinterpret_cast<float2*>(ws + s.part_ml);
  a.out = static_cast<uint16_t*>(k.out);
  const int rc = status_of(launch_qcache_queries(r, a, st));
  return rc ? rc : status_of(launch_qcache_attn(a, st));
}

}  // namespace
}  // namespace sv

using namespace sv;

extern "C" {

int spec_rope_frequencies(const spec_rope_config* r, int head_dim, double* out) {
  return out ? rope_frequencies(r, head_dim, out) : SPEC_EINVAL;
}

int spec_rope(const spec_rope_config* r, int dtype, const void* x, int64_t x_row_stride,
              int64_t x_head_stride, void* out, int64_t out_row_stride, int64_t out_head_stride,
              const int32_t* positions, int n_rows, int n_heads, int head_dim, int inverse,
              void* stream) {
  if (!r || !x || !out || !positions || n_rows < 1 || n_heads < 1) return SPEC_EINVAL;
  if (dtype != SPEC_BF16 && dtype != SPEC_FP16 && dtype != SPEC_FP32) return SPEC_EINVAL;
  RopeArgs ra;
  const int rc = rope_args(r, head_dim, &ra);
  if (rc) return rc;
  const size_t size = dtype == SPEC_FP32 ? 4 : 2;
  if (!aligned(x, size) || !aligned(out, size)) return SPEC_EINVAL;
  if (x_row_stride < 0 || x_head_stride < 0 || out_row_stride < 0 || out_head_stride < 0) return SPEC_EINVAL;
  // the written heads and rows must be apart, in either order of nesting
  const bool by_row = (n_heads == 1 || out_head_stride >= head_dim) &&
                      (n_rows == 1 || out_row_stride >= (__int128)(n_heads - 1) * out_head_stride + head_dim);
  const bool by_head = (n_rows == 1 || out_row_stride >= head_dim) &&
                       (n_heads == 1 || out_head_stride >= (__int128)(n_rows - 1) * out_row_stride + head_dim);
  if (!by_row && !by_head) return SPEC_EINVAL;
  if (x == out && ((n_rows > 1 && x_row_stride != out_row_stride) ||
                   (n_heads > 1 && x_head_stride != out_head_stride)))
    return SPEC_EINVAL;
  RopeOpArgs a{};
  a.x = x;
  a.out = out;
  a.x_row = x_row_stride;
  a.x_head = x_head_stride;
  a.out_row = out_row_stride;
  a.out_head = out_head_stride;
  a.positions = positions;
  a.n_rows = n_rows;
  a.n_heads = n_heads;
  a.dim = head_dim;
  a.inverse = inverse;
  return status_of(launch_rope(ra, a, dtype, static_cast<cudaStream_t>(stream)));
}

size_t spec_qcache_write_workspace_bytes(const spec_qcache* c, int max_batch, int max_n) {
  if (check_cache(c) || max_batch < 1 || max_n < 0 || max_n > SPEC_QCACHE_MAX_WRITE) return 0;
  return kWsHeaderBytes;
}

int spec_qcache_write(const spec_qcache* c, const spec_rope_config* r, const int32_t* block_table,
                      int max_pages, const int32_t* seq_lens, int B, int n, const void* k_new,
                      int64_t k_row_stride, const void* v_new, int64_t v_row_stride, void* ws,
                      size_t ws_bytes, void* stream) {
  int rc = check_cache(c);
  if (rc) return rc;
  RopeArgs ra;
  rc = rope_args(r, c->head_dim, &ra);
  if (rc) return rc;
  rc = check_write(c, block_table, max_pages, seq_lens, B, n, k_new, k_row_stride, v_new, v_row_stride);
  if (rc) return rc;
  if (!ws || ws_bytes < kWsHeaderBytes || !aligned(ws, 256)) return SPEC_EINVAL;
  if (n == 0) return SPEC_OK;
  return run_write(c, ra, block_table, max_pages, seq_lens, B, n, k_new, k_row_stride, v_new,
                   v_row_stride, ws, static_cast<cudaStream_t>(stream));
}

size_t spec_qcache_attn_workspace_bytes(const spec_qcache* c, int n_q_heads, int max_batch, int max_n,
                                        int max_pages, int window) {
  if (check_cache(c)) return 0;
  return attn_bytes(c, n_q_heads, max_batch, max_n, max_pages, window);
}

int spec_qcache_attn(const spec_qcache* c, const spec_rope_config* r, const void* q,
                     int64_t q_row_stride, int n_q_heads, const int32_t* block_table, int max_pages,
                     const int32_t* seq_lens, int B, int n, int q_offset, int kv_extra, int window,
                     float scale, void* out, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_cache(c);
  if (rc) return rc;
  RopeArgs ra;
  rc = rope_args(r, c->head_dim, &ra);
  if (rc) return rc;
  const AttnCall k{q, q_row_stride, n_q_heads, block_table, max_pages, seq_lens, B, n, q_offset,
                   kv_extra, window, scale, out, ws, ws_bytes};
  AttnLayout s;
  rc = check_attn(c, k, &s);
  return rc ? rc : run_attn(c, ra, k, s, static_cast<cudaStream_t>(stream));
}

int spec_qcache_verify_attn(const spec_qcache* c, const spec_rope_config* r, const void* q,
                            int64_t q_row_stride, int n_q_heads, const void* k_new,
                            int64_t k_row_stride, const void* v_new, int64_t v_row_stride,
                            const int32_t* block_table, int max_pages, const int32_t* seq_lens,
                            int B, int n, int window, float scale, void* out, void* ws,
                            size_t ws_bytes, void* stream) {
  int rc = check_cache(c);
  if (rc) return rc;
  RopeArgs ra;
  rc = rope_args(r, c->head_dim, &ra);
  if (rc) return rc;
  rc = check_write(c, block_table, max_pages, seq_lens, B, n, k_new, k_row_stride, v_new, v_row_stride);
  if (rc) return rc;
  const AttnCall k{q, q_row_stride, n_q_heads, block_table, max_pages, seq_lens, B, n, 0,
                   n, window, scale, out, ws, ws_bytes};
  AttnLayout s;
  rc = check_attn(c, k, &s);
  if (rc) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  rc = run_write(c, ra, block_table, max_pages, seq_lens, B, n, k_new, k_row_stride, v_new,
                 v_row_stride, ws, st);
  return rc ? rc : run_attn(c, ra, k, s, st);
}

}  // extern "C"
