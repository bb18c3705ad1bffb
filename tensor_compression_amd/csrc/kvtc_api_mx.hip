// C ABI of the microscaled paged cache: argument checks, the split of the
// attention over workgroups, and the launch sequences.
#include <math.h>

#include <algorithm>
#include <utility>

#include "mx_internal.h"

using namespace kvtc;

namespace {

constexpr int64_t kMaxGrid = (1 << 24) - 1;  // workgroups of 256 threads in a launch

bool misaligned(const void* p, unsigned to = 16) { return ((uintptr_t)p & (to - 1)) != 0; }

// Whether n 4-byte words at a and m at b share any.
bool overlap(const void* a, int64_t n, const void* b, int64_t m) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && x < y + 4 * (uint64_t)m && y < x + 4 * (uint64_t)n;
}

// n rows of `bytes` bytes, `stride` bytes apart, and whether any of two such
// tensors share a byte.
struct RowBytes {
  const void* at;
  int64_t bytes, stride, n;
};
bool meet(RowBytes a, RowBytes b) {
  for (RowBytes* x : {&a, &b})
    if (x->n > 1 && x->stride <= x->bytes) {  // without gaps
      x->bytes += (x->n - 1) * x->stride;
      x->n = 1;
    }
  if (a.n < b.n) std::swap(a, b);
  typedef __int128 wide;
  const wide d = (wide)(uintptr_t)b.at - (wide)(uintptr_t)a.at;
  if (d >= (wide)a.stride * (a.n - 1) + a.bytes || -d >= (wide)b.stride * (b.n - 1) + b.bytes) return false;
  // row i of a meets one at x where x - a.bytes < i a.stride < x + b.bytes
  auto some = [&](wide x, int64_t first, int64_t last) {
    if (a.n == 1) return x < a.bytes && -x < b.bytes;
    const wide low = x - a.bytes, i = low / a.stride - (low % a.stride < 0) + 1;
    return std::max<wide>(i, first) <= last && std::max<wide>(i, first) * a.stride < x + b.bytes;
  };
  if (a.stride == b.stride) return some(d, 1 - b.n, a.n - 1);  // rows i and j: as i - j and 0
  for (int64_t j = 0; j < b.n; ++j)
    if (some(d + (wide)j * b.stride, 0, a.n - 1)) return true;
  return false;
}

kvtc_status check_config(const kvtc_mx_config* c) {
  if (!c) return KVTC_ERR_INVALID_ARG;
  if (c->layers < 1 || c->kv_heads < 1 || c->pool_pages < 1) return KVTC_ERR_INVALID_ARG;
  if (c->dtype != KVTC_BF16 && c->dtype != KVTC_FP32) return KVTC_ERR_INVALID_ARG;
  if ((c->bits_k != 4 && c->bits_k != 8) || (c->bits_v != 4 && c->bits_v != 8)) return KVTC_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return KVTC_ERR_UNSUPPORTED;
  if ((int64_t)c->layers * c->kv_heads > 65536) return KVTC_ERR_UNSUPPORTED;
  return KVTC_OK;
}

int64_t layer_bytes(const kvtc_mx_config& c) {
  return (int64_t)c.pool_pages * c.kv_heads * mx_record(c.head_dim, c.bits_k, c.bits_v).bytes;
}

kvtc_status check_batch(const kvtc_mx_batch* b) {
  if (!b || b->reserved != 0) return KVTC_ERR_INVALID_ARG;
  if (b->n_seqs < 0 || b->max_pages < 1 || b->total_rows < 0 || b->max_rows < 0 || b->max_len < 0)
    return KVTC_ERR_INVALID_ARG;
  if ((int64_t)b->max_len > (int64_t)b->max_pages * KVTC_MX_PAGE || b->max_len > (1 << 30)) return KVTC_ERR_INVALID_ARG;
  if (b->n_seqs > 0 && (!b->page_table || !b->kv_lens || !b->row_start)) return KVTC_ERR_INVALID_ARG;
  if (misaligned(b->page_table, 4) || misaligned(b->kv_lens, 4) || misaligned(b->row_start, 4))
    return KVTC_ERR_INVALID_ARG;
  return KVTC_OK;
}

bool nothing_to_do(const kvtc_mx_batch& b) { return b.n_seqs == 0 || b.total_rows == 0 || b.max_rows == 0; }

// Configuration, batch, pool and status, common to every call; *layer is the
// first record of `layer`.
kvtc_status check_call(const kvtc_mx_config* cfg, const kvtc_mx_batch* batch, int32_t layer, int32_t n_layers,
                       const void* pool, size_t pool_bytes, const uint32_t* status, uint8_t** first) {
  kvtc_status st = check_config(cfg);
  if (st != KVTC_OK) return st;
  st = check_batch(batch);
  if (st != KVTC_OK) return st;
  if (layer < 0 || n_layers < 1 || n_layers > cfg->layers || layer > cfg->layers - n_layers) return KVTC_ERR_INVALID_ARG;
  if (!pool || misaligned(pool) || misaligned(status, 4)) return KVTC_ERR_INVALID_ARG;
  if (pool_bytes / (size_t)cfg->layers < (size_t)layer_bytes(*cfg)) return KVTC_ERR_CAPACITY;
  *first = (uint8_t*)const_cast<void*>(pool) + layer * layer_bytes(*cfg);
  return KVTC_OK;
}

// Strides of a row tensor: whole 16 bytes, none negative; of an output also
// such that no two elements fall together (each stride passes the span of
// the smaller ones).
bool bad_strides(const int64_t* st, const int64_t (&extent)[3], int D, int elem, bool out) {
  if (!st) return true;
  for (int i = 0; i < 3; ++i)
    if (st[i] < 0 || st[i] > ((int64_t)1 << 46) || (st[i] * elem) % 16) return true;
  if (!out) return false;
  std::pair<int64_t, int64_t> d[3];
  for (int i = 0; i < 3; ++i) d[i] = {st[i], extent[i]};
  std::sort(d, d + 3);
  __int128 span = D;  // 2^46 by 2^31 rows passes 64 bits
  for (const auto& [s, n] : d) {
    if (n < 2) continue;
    if (s < span) return true;
    span += (__int128)s * (n - 1);
  }
  return false;
}

// Checks of a write or read, and its parameters but for the units.
kvtc_status io_params(const kvtc_mx_config* cfg, const kvtc_mx_batch* b, int32_t layer, int32_t n_layers, void* k,
                      const int64_t* ks, void* v, const int64_t* vs, const void* pool, size_t pool_bytes, int32_t dtype,
                      uint32_t* status, bool write, MxIoParams* p) {
  uint8_t* first;
  const kvtc_status st = check_call(cfg, b, layer, n_layers, pool, pool_bytes, status, &first);
  if (st != KVTC_OK) return st;
  if (dtype != KVTC_BF16 && dtype != KVTC_FP32) return KVTC_ERR_INVALID_ARG;
  const int64_t extent[3] = {n_layers, cfg->kv_heads, b->total_rows};
  const int elem = dtype == KVTC_BF16 ? 2 : 4;
  if (bad_strides(ks, extent, cfg->head_dim, elem, !write) || bad_strides(vs, extent, cfg->head_dim, elem, !write))
    return KVTC_ERR_INVALID_ARG;
  if (!nothing_to_do(*b) && (!k || !v || misaligned(k) || misaligned(v))) return KVTC_ERR_INVALID_ARG;
  p->b = *b;
  p->H = cfg->kv_heads;
  p->pool_pages = cfg->pool_pages;
  p->n_layers = n_layers;
  p->pool = first;
  p->layer_bytes = layer_bytes(*cfg);
  p->x[0] = k;
  p->x[1] = v;
  for (int i = 0; i < 3; ++i) {
    p->st[0][i] = ks[i];
    p->st[1][i] = vs[i];
  }
  p->status = status;
  return KVTC_OK;
}

kvtc_status io_call(const kvtc_mx_config* cfg, const kvtc_mx_batch* b, int32_t layer, int32_t n_layers, void* k,
                    const int64_t* ks, void* v, const int64_t* vs, const void* pool, size_t pool_bytes, int32_t dtype,
                    uint32_t* status, bool write, hipStream_t stream) {
  MxIoParams p{};
  const kvtc_status st =
      io_params(cfg, b, layer, n_layers, k, ks, v, vs, pool, pool_bytes, dtype, status, write, &p);
  if (st != KVTC_OK || nothing_to_do(*b)) return st;
  // n rows that start anywhere in a page touch at most ceil((n + 15) / 16) pages
  const int64_t rows = std::min({b->max_rows, b->total_rows, b->max_len});
  const int64_t units = std::max<int64_t>((rows + 2 * KVTC_MX_PAGE - 2) / KVTC_MX_PAGE, 1);
  if (units * b->n_seqs > kMaxGrid) return KVTC_ERR_UNSUPPORTED;
  p.n_units = (int32_t)units;
  const hipError_t e = write ? launch_mx_write(p, cfg->head_dim, cfg->bits_k, cfg->bits_v, dtype == KVTC_FP32, stream)
                             : launch_mx_read(p, cfg->head_dim, cfg->bits_k, cfg->bits_v, dtype == KVTC_FP32, stream);
  return e == hipSuccess ? KVTC_OK : KVTC_ERR_HIP;
}

kvtc_status check_rope(const kvtc_mx_rope* r, int D, MxRopeParams* p) {
  if (!r || r->reserved != 0) return KVTC_ERR_INVALID_ARG;
  if (r->style != KVTC_ROPE_HALF && r->style != KVTC_ROPE_INTERLEAVED) return KVTC_ERR_INVALID_ARG;
  if (r->rot_dim < 2 || r->rot_dim > D || r->axes < 1 || r->axes > 4) return KVTC_ERR_INVALID_ARG;
  if (r->rot_dim % 16) return KVTC_ERR_UNSUPPORTED;  // a lane's channels would be of both halves
  if (!r->freqs || misaligned(r->freqs, 8)) return KVTC_ERR_INVALID_ARG;
  for (int j = 0; r->axis && j < r->rot_dim / 2; ++j) {
    if (r->axis[j] >= r->axes) return KVTC_ERR_INVALID_ARG;
    p->axis[j / 32] |= (uint64_t)r->axis[j] << (2 * (j % 32));
  }
  p->freqs = r->freqs;
  p->rot = r->rot_dim;
  p->interleaved = r->style == KVTC_ROPE_INTERLEAVED;
  return KVTC_OK;
}

// Masks of drafts: [total_rows][words].
kvtc_status check_masks(const kvtc_mx_batch& b, const uint32_t* masks, int32_t words) {
  if (words < 1 || (int64_t)words * 32 < b.max_rows) return KVTC_ERR_INVALID_ARG;
  if (b.max_rows > KVTC_MX_MAX_DRAFT || words > KVTC_MX_MAX_DRAFT / 32) return KVTC_ERR_UNSUPPORTED;
  if (misaligned(masks, 4) || (!masks && !nothing_to_do(b))) return KVTC_ERR_INVALID_ARG;
  return KVTC_OK;
}

// How one pass of the attention is cut up.
struct Cut {
  int nt;             // 16-row tiles of a workgroup: 1 or 2 (k_mx_attn), 8 (k_mx_rows)
  int waves;          // waves of a workgroup
  int64_t tiles;      // workgroups along the rows
  int nsplit, chunk;  // workgroups along the tokens, tokens of each
};
Cut cut_pass(int64_t rows, int64_t seqs, int H, int64_t span) {
  Cut c{};
  c.nt = rows <= 16 ? 1 : rows <= 64 ? 2 : 8;
  c.tiles = (rows + 16 * c.nt - 1) / (16 * c.nt);
  // As many workgroups as the card takes at its rate: one a CU for few rows
  // (1 sequence of 131072 tokens: 41 us with 256, 42 with 768, and more
  // partials to join), two for many rows, which need the second's waves (128
  // sequences behind 32768 tokens: 220 us with 256, 166 with 512) unless
  // that left them less than 512 tokens each (64 behind 8192: 25 us and 6 for
  // the join, with ranges of 256 29 and 8).
  const int64_t units = c.tiles * H * seqs, room = c.nt == 8 ? 512 : 256;
  int64_t n = std::max<int64_t>(1, std::min(room / units, c.nt == 8 ? span / 512 : (span + 127) / 128));
  // A second launch and its join cost about 3 us, what a workgroup takes for
  // 800 tokens (16 sequences of 1000 tokens: whole 8.2, halved 9.7 us; 1
  // sequence of 1000: whole 7.9, in eight 7.3 us).
  if (c.nt != 8 && span - span / n <= 800) n = 1;
  c.chunk = (int)(((span + n - 1) / n + 127) / 128 * 128);
  c.nsplit = (int)std::max<int64_t>(1, (span + c.chunk - 1) / std::max(c.chunk, 1));
  // Eight waves where a CU has one workgroup with enough for all of them (24
  // sequences of 16000 tokens: 114 -> 79 us; the prefix of 4 sequences behind
  // 131072: 47 -> 41); beside others, or with little to do, four (40 of 4000:
  // 34 us, eight 40; 1 of 8000 in 256s: 8.7 and 9.0).
  c.waves = c.nt == 1 && units <= 256 && c.chunk > 512 ? 8 : 4;
  return c;
}

struct AttnPlan {
  Cut prefix, own;  // nsplit 0: no such pass
  int begin;        // first token of `own`
  bool once;        // `own` reads its codes past the caches
  bool together;    // both in one launch
  int64_t slots, ws;
};

kvtc_status plan_attn(const kvtc_mx_config& c, const kvtc_mx_batch& b, int32_t q_heads, int32_t shared, bool tree,
                      AttnPlan* a) {
  if (q_heads < c.kv_heads || q_heads % c.kv_heads) return KVTC_ERR_INVALID_ARG;
  if (shared < 0 || shared > b.max_pages) return KVTC_ERR_INVALID_ARG;
  if ((int64_t)b.total_rows * q_heads > 0x7FFFFFFF) return KVTC_ERR_UNSUPPORTED;
  *a = AttnPlan{};
  if (nothing_to_do(b)) return KVTC_OK;
  const int G = q_heads / c.kv_heads;
  a->begin = (int)std::min<int64_t>((int64_t)shared * KVTC_MX_PAGE, b.max_len);
  const int64_t rows = (int64_t)std::min(b.max_rows, b.total_rows) * G;
  if (a->begin < b.max_len || a->begin == 0) a->own = cut_pass(rows, b.n_seqs, c.kv_heads, b.max_len - a->begin);
  // at most this many bytes of codes (past 64 bits in calls that are refused
  // below), against the 256 MB of the memory-side cache
  a->once = (double)b.n_seqs * (b.max_len - a->begin) / KVTC_MX_PAGE * c.kv_heads *
                mx_record(c.head_dim, c.bits_k, c.bits_v).bytes > 0x1p28;
  if (a->begin > 0) {
    a->prefix = cut_pass((int64_t)b.total_rows * G, 1, c.kv_heads, a->begin);
    // One launch where the prefix takes the kernel for many rows and the own
    // tokens the one for few (64 sequences of 1000 own tokens behind 2048: 40
    // us one after the other, 29 together; 128 of 1800 behind 8192: 100 and
    // 98).  Codes past the caches go one after the other: the shared kernel's
    // registers leave the own tokens 2 waves a SIMD instead of 3 (4 bits: 64
    // of 8000 behind 32768 173 us together, 156 so, 128 of 4000 behind 8192
    // 158 and 145; 8 bits, with half the instructions a byte, would take it
    // the other way behind short prefixes: 64 of 4000 behind 8192 121 and 136,
    // behind 32768 171 and 167).  Four waves a workgroup beside the prefix's
    // (20 of 4000 behind 8192: 41 us, in a launch of eight 51), otherwise as
    // `cut_pass` says (8 of 16000 behind 1024: 48 -> 42 us, 24 of 16000 behind
    // 8192: 140 -> 103).
    a->together = a->prefix.nt == 8 && a->own.nt == 1 && !a->once;
    if (a->together) a->own.waves = 4;
    // Drafts: also where both take the kernel for many rows (32 sequences of 10
    // to 25 rows behind 8192: 125 us a call one after the other, 109 so; fp32
    // 260 and 230).  Rows without masks were not timed this way, and have no
    // such kernel.
    if (tree && a->prefix.nt == 8 && a->own.nt == 8 &&
        (a->own.tiles * a->own.nsplit * b.n_seqs + a->prefix.tiles * a->prefix.nsplit) * c.kv_heads <= kMaxGrid)
      a->together = true;
  }
  a->slots = a->begin > 0 || a->own.nsplit > 1 ? a->prefix.nsplit + a->own.nsplit : 0;
  a->ws = a->slots * b.total_rows * q_heads * (int64_t)(c.head_dim + 2) * 4;
  // (each its own launch; in one, own tokens on 16-row tiles have at most 256
  // MB of codes, so fewer than 2^22 workgroups, and the prefix 2^20; the
  // drafts' 128-row tiles of both were added up above)
  if (a->own.tiles * c.kv_heads * std::max(a->own.nsplit, 1) * b.n_seqs > kMaxGrid ||
      a->prefix.tiles * c.kv_heads * std::max(a->prefix.nsplit, 1) > kMaxGrid ||
      (int64_t)b.total_rows * q_heads > 4 * kMaxGrid)
    return KVTC_ERR_UNSUPPORTED;
  return KVTC_OK;
}

// masks: rows are drafts (then causal is 0).
kvtc_status attn_call(const kvtc_mx_config* cfg, const kvtc_mx_batch* b, int32_t layer, const void* pool,
                      size_t pool_bytes, int32_t shared, const uint32_t* masks, int32_t words, const void* q,
                      int64_t q_stride, int32_t q_heads, float scale, int32_t causal, void* out, float* lse, void* ws,
                      size_t ws_bytes, uint32_t* status, hipStream_t stream) {
  uint8_t* first;
  kvtc_status st = check_call(cfg, b, layer, 1, pool, pool_bytes, status, &first);
  if (st != KVTC_OK) return st;
  AttnPlan a;
  st = plan_attn(*cfg, *b, q_heads, shared, masks != nullptr, &a);
  if (st != KVTC_OK) return st;
  const int elem = cfg->dtype == KVTC_BF16 ? 2 : 4;
  if (!(scale > 0.0f && scale <= 0x1p100f) || !isnormal(scale) || (causal != 0 && causal != 1)) return KVTC_ERR_INVALID_ARG;
  if (q_stride < 0 || q_stride > ((int64_t)1 << 46) || (q_stride * elem) % 16) return KVTC_ERR_INVALID_ARG;
  if (nothing_to_do(*b)) return KVTC_OK;
  if (!q || !out || misaligned(q) || misaligned(out) || misaligned(lse, 4) || misaligned(ws)) return KVTC_ERR_INVALID_ARG;
  if (a.ws > 0 && !ws) return KVTC_ERR_INVALID_ARG;
  if ((int64_t)ws_bytes < a.ws) return KVTC_ERR_CAPACITY;
  const bool f32 = cfg->dtype == KVTC_FP32;
  MxAttnParams p{};
  p.b = *b;
  p.pool = first;
  p.pool_pages = cfg->pool_pages;
  p.H = cfg->kv_heads;
  p.G = q_heads / cfg->kv_heads;
  p.q = q;
  p.q_stride = q_stride;
  p.c = (float)((double)scale * 1.4426950408889634);
  p.causal = causal;
  p.out = out;
  p.lse = lse;
  p.status = status;
  p.masks = masks;
  p.words = words;
  if (a.slots) {
    p.ws_o = (float*)ws;
    p.ws_ml = (float2*)(p.ws_o + a.slots * b->total_rows * q_heads * (int64_t)cfg->head_dim);
  }
  auto cut = [&](const Cut& c) {
    p.nt = c.nt;
    p.waves = c.waves;
    p.tiles = (int32_t)c.tiles;
    p.nsplit = c.nsplit;
    p.chunk = c.chunk;
  };
  cut(a.prefix);
  p.prefix = 1;
  p.end = a.begin;
  const MxAttnParams prefix = p;
  cut(a.own);
  p.prefix = 0;
  p.begin = a.begin;
  p.end = 0x7FFFFFFF;
  p.slot0 = a.prefix.nsplit;
  p.fold = causal && a.own.nt == 8 && a.own.tiles * cfg->kv_heads * a.own.nsplit * b->n_seqs <= 512;
  // Whole sequences, more workgroups than compute units: first the longest, one
  // a unit and in rising order, then the others from the longest on, so that
  // the second of a unit makes up for its first (sequences of 511 to 8191
  // tokens, 8 heads: 64 of them 67 -> 62 us, 128 115 -> 94, with 5 rows each
  // 89 -> 79 and 146 -> 120; all of 4000: 64 46.7 -> 47.7, so not where they
  // are short).
  const int64_t per_round = std::max(256 / cfg->kv_heads, 1);
  if (!a.prefix.nsplit && a.own.nt < 8 && a.own.tiles == 1 && a.own.nsplit == 1 && b->n_seqs > per_round &&
      b->n_seqs <= 256 && b->max_len >= 2048)
    p.pair = (int32_t)per_round;
  // Drafts in two tiles of 32 rows, more workgroups than the card holds at once
  // (two a unit): the longest sequences first (64 of 511 to 8191 tokens, 5 to
  // 16 rows of 4 heads each: 141 -> 112 us).  The longest takes as long as the
  // call (8064 tokens, an even share is 6795).  Rows without masks were not
  // timed in this order, and keep that of the batch.
  if (masks && !a.prefix.nsplit && a.own.nt == 2 && a.own.tiles > 1 && a.own.nsplit == 1 &&
      a.own.tiles * cfg->kv_heads * b->n_seqs > 512 && b->n_seqs <= 256 && b->max_len >= 2048)
    p.pair = 1;
  p.once = a.once;
  p.together = a.together;
  const auto launch = masks ? launch_mx_attn_tree : launch_mx_attn;
  if (launch(a.prefix.nsplit ? &prefix : nullptr, a.own.nsplit ? &p : nullptr, cfg->head_dim, cfg->bits_k, cfg->bits_v,
             f32, stream) != hipSuccess)
    return KVTC_ERR_HIP;
  if (!a.slots) return KVTC_OK;
  MxJoinParams j{};
  j.b = *b;
  j.Hq = q_heads;
  j.D = cfg->head_dim;
  j.causal = causal;
  j.begin = a.begin;
  j.prefix_splits = a.prefix.nsplit;
  j.prefix_chunk = a.prefix.chunk;
  j.nsplit = a.own.nsplit;
  j.chunk = std::max(a.own.chunk, 1);
  j.ws_o = p.ws_o;
  j.ws_ml = p.ws_ml;
  j.out = out;
  j.lse = lse;
  j.status = status;
  return launch_mx_join(j, f32, stream) == hipSuccess ? KVTC_OK : KVTC_ERR_HIP;
}

kvtc_status attn_workspace(const kvtc_mx_config* cfg, const kvtc_mx_batch* batch, int32_t q_heads, int32_t shared_pages,
                           bool tree, size_t* ws_bytes) {
  kvtc_status st = check_config(cfg);
  if (st == KVTC_OK) st = check_batch(batch);
  if (st != KVTC_OK) return st;
  if (!ws_bytes) return KVTC_ERR_INVALID_ARG;
  AttnPlan a;
  st = plan_attn(*cfg, *batch, q_heads, shared_pages, tree, &a);
  if (st == KVTC_OK) *ws_bytes = (size_t)a.ws;
  return st;
}

}  // namespace

extern "C" {

kvtc_status kvtc_mx_pool_size(const kvtc_mx_config* cfg, size_t* record_bytes, size_t* pool_bytes) {
  const kvtc_status st = check_config(cfg);
  if (st != KVTC_OK) return st;
  if (!record_bytes || !pool_bytes) return KVTC_ERR_INVALID_ARG;
  *record_bytes = (size_t)mx_record(cfg->head_dim, cfg->bits_k, cfg->bits_v).bytes;
  *pool_bytes = (size_t)cfg->layers * (size_t)layer_bytes(*cfg);
  return KVTC_OK;
}

kvtc_status kvtc_mx_write(const kvtc_mx_config* cfg, const kvtc_mx_batch* batch, int32_t layer, int32_t n_layers,
                          const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides,
                          void* pool, size_t pool_bytes, uint32_t* status_dev, hipStream_t stream) {
  return io_call(cfg, batch, layer, n_layers, const_cast<void*>(k), k_strides, const_cast<void*>(v), v_strides, pool,
                 pool_bytes, cfg ? cfg->dtype : 0, status_dev, true, stream);
}

kvtc_status kvtc_mx_read(const kvtc_mx_config* cfg, const kvtc_mx_batch* batch, int32_t layer, int32_t n_layers,
                         const void* pool, size_t pool_bytes, void* k_out, const int64_t* k_strides, void* v_out,
                         const int64_t* v_strides, int32_t out_dtype, uint32_t* status_dev, hipStream_t stream) {
  return io_call(cfg, batch, layer, n_layers, k_out, k_strides, v_out, v_strides, pool, pool_bytes, out_dtype,
                 status_dev, false, stream);
}

kvtc_status kvtc_mx_attn_workspace(const kvtc_mx_config* cfg, const kvtc_mx_batch* batch, int32_t q_heads,
                                   int32_t shared_pages, size_t* ws_bytes) {
  return attn_workspace(cfg, batch, q_heads, shared_pages, false, ws_bytes);
}

kvtc_status kvtc_mx_attn(const kvtc_mx_config* cfg, const kvtc_mx_batch* batch, int32_t layer, const void* pool,
                         size_t pool_bytes, const void* q, int64_t q_stride, int32_t q_heads, float scale,
                         int32_t causal, void* out, float* lse, void* ws, size_t ws_bytes, uint32_t* status_dev,
                         hipStream_t stream) {
  return attn_call(cfg, batch, layer, pool, pool_bytes, 0, nullptr, 0, q, q_stride, q_heads, scale, causal, out, lse, ws, ws_bytes,
                   status_dev, stream);
}

kvtc_status kvtc_mx_attn_shared(const kvtc_mx_config* cfg, const kvtc_mx_batch* batch, int32_t layer,
                                const void* pool, size_t pool_bytes, int32_t shared_pages, const void* q,
                                int64_t q_stride, int32_t q_heads, float scale, int32_t causal, void* out, float* lse,
                                void* ws, size_t ws_bytes, uint32_t* status_dev, hipStream_t stream) {
  return attn_call(cfg, batch, layer, pool, pool_bytes, shared_pages, nullptr, 0, q, q_stride, q_heads, scale, causal, out, lse,
                   ws, ws_bytes, status_dev, stream);
}

kvtc_status kvtc_mx_write_rope(const kvtc_mx_config* cfg, const kvtc_mx_batch* batch, int32_t layer, int32_t n_layers,
                               const kvtc_mx_rope* rope, const int32_t* positions, const void* k,
                               const int64_t* k_strides, const void* v, const int64_t* v_strides, const void* q,
                               int64_t q_stride, int32_t q_heads, void* q_out, int64_t q_out_stride, void* pool,
                               size_t pool_bytes, uint32_t* status_dev, hipStream_t stream) {
  MxRopeParams p{};
  kvtc_status st = io_params(cfg, batch, layer, n_layers, const_cast<void*>(k), k_strides, const_cast<void*>(v),
                             v_strides, pool, pool_bytes, cfg ? cfg->dtype : 0, status_dev, true, &p.io);
  if (st != KVTC_OK) return st;
  st = check_rope(rope, cfg->head_dim, &p);
  if (st != KVTC_OK) return st;
  if (misaligned(positions, 4) || (!positions && rope->axes != 1)) return KVTC_ERR_INVALID_ARG;
  if (q_heads < 0 || (q_heads > 0 && n_layers != 1)) return KVTC_ERR_INVALID_ARG;
  const int elem = cfg->dtype == KVTC_BF16 ? 2 : 4;
  if (q_heads > 0) {
    for (const int64_t s : {q_stride, q_out_stride})
      if (s < 0 || s > ((int64_t)1 << 46) || (s * elem) % 16) return KVTC_ERR_INVALID_ARG;
    if (batch->total_rows > 1 && q_out_stride < (int64_t)q_heads * cfg->head_dim) return KVTC_ERR_INVALID_ARG;
  }
  if (nothing_to_do(*batch)) return KVTC_OK;
  if (q_heads > 0 && (!q || !q_out || misaligned(q) || misaligned(q_out) || (q == q_out && q_stride != q_out_stride)))
    return KVTC_ERR_INVALID_ARG;
  auto slices = [](int64_t n) { return (n + kMxRopeSlice - 1) / kMxRopeSlice; };
  const int64_t parts = 2 * slices(cfg->kv_heads) + slices(q_heads);
  p.positions = positions;
  p.Hq = q_heads;
  p.parts = (int32_t)parts;
  p.q = q;
  p.q_out = q_out;
  p.q_stride = q_stride;
  p.q_out_stride = q_out_stride;
  // (queries of rows before the first token too, so max_len is no bound here)
  const int64_t rows = std::min(batch->max_rows, batch->total_rows);
  const int64_t units = std::max<int64_t>((rows + 2 * KVTC_MX_PAGE - 2) / KVTC_MX_PAGE, 1);
  if (units * batch->n_seqs > kMaxGrid || parts * n_layers > 65535) return KVTC_ERR_UNSUPPORTED;
  if (q_heads > 0) {  // what other workgroups still read
    const int64_t D = cfg->head_dim * elem, n = batch->total_rows;
    const RowBytes to{q_out, q_heads * D, q_out_stride * elem, n};
    auto over = [&](const void* x, int64_t bytes) { return x && meet(to, RowBytes{x, bytes, 0, 1}); };
    bool bad = (q != q_out && meet(to, RowBytes{q, q_heads * D, q_stride * elem, n})) || over(positions, n * rope->axes * 4) ||
               over(rope->freqs, rope->rot_dim * 4) || over(batch->page_table, (int64_t)batch->n_seqs * batch->max_pages * 4) ||
               over(batch->kv_lens, (int64_t)batch->n_seqs * 4) || over(batch->row_start, ((int64_t)batch->n_seqs + 1) * 4) ||
               over(pool, cfg->layers * layer_bytes(*cfg));
    for (int i = 0; i < 2; ++i) {
      const int64_t head = p.io.st[i][1] * elem, row = p.io.st[i][2] * elem;
      const int heads = head == D ? 1 : cfg->kv_heads;  // side by side: as one
      for (int h = 0; h < heads; ++h)
        bad |= meet(to, RowBytes{(const uint8_t*)p.io.x[i] + h * head, D * (cfg->kv_heads / heads), row, n});
    }
    if (bad) return KVTC_ERR_INVALID_ARG;
  }
  p.io.n_units = (int32_t)units;
  return launch_mx_rope(p, cfg->head_dim, cfg->bits_k, cfg->bits_v, cfg->dtype == KVTC_FP32, stream) == hipSuccess
             ? KVTC_OK
             : KVTC_ERR_HIP;
}

kvtc_status kvtc_mx_tree(const kvtc_mx_batch* batch, const int32_t* parents, uint32_t* masks, int32_t words,
                         int32_t* positions, uint32_t* status_dev, hipStream_t stream) {
  kvtc_status st = check_batch(batch);
  if (st == KVTC_OK) st = check_masks(*batch, masks, words);
  if (st != KVTC_OK) return st;
  if (misaligned(parents, 4) || misaligned(positions, 4) || misaligned(status_dev, 4)) return KVTC_ERR_INVALID_ARG;
  if (nothing_to_do(*batch)) return KVTC_OK;
  if (!parents) return KVTC_ERR_INVALID_ARG;
  if (batch->n_seqs > kMaxGrid) return KVTC_ERR_UNSUPPORTED;
  // several waves read the parents, lengths and rows while others write
  const int64_t rows = batch->total_rows, n = batch->n_seqs;
  auto apart = [&](const void* out, int64_t words_out) {
    return !overlap(out, words_out, parents, rows) && !overlap(out, words_out, batch->kv_lens, n) &&
           !overlap(out, words_out, batch->row_start, n + 1);
  };
  if (!apart(positions, rows) || !apart(masks, rows * words) || overlap(positions, rows, masks, rows * words))
    return KVTC_ERR_INVALID_ARG;
  return launch_mx_tree(*batch, parents, masks, words, positions, status_dev, stream) == hipSuccess ? KVTC_OK
                                                                                                  : KVTC_ERR_HIP;
}

kvtc_status kvtc_mx_attn_tree_workspace(const kvtc_mx_config* cfg, const kvtc_mx_batch* batch, int32_t q_heads,
                                        int32_t shared_pages, size_t* ws_bytes) {
  return attn_workspace(cfg, batch, q_heads, shared_pages, true, ws_bytes);
}

kvtc_status kvtc_mx_attn_tree(const kvtc_mx_config* cfg, const kvtc_mx_batch* batch, int32_t layer, const void* pool,
                              size_t pool_bytes, int32_t shared_pages, const uint32_t* masks, int32_t words,
                              const void* q, int64_t q_stride, int32_t q_heads, float scale, void* out, float* lse,
                              void* ws, size_t ws_bytes, uint32_t* status_dev, hipStream_t stream) {
  kvtc_status st = check_config(cfg);
  if (st == KVTC_OK) st = check_batch(batch);
  if (st == KVTC_OK) st = check_masks(*batch, masks, words);
  if (st != KVTC_OK) return st;
  return attn_call(cfg, batch, layer, pool, pool_bytes, shared_pages, masks, words, q, q_stride, q_heads, scale, 0, out,
                   lse, ws, ws_bytes, status_dev, stream);
}

kvtc_status kvtc_mx_keep(const kvtc_mx_config* cfg, const kvtc_mx_batch* batch, int32_t layer, int32_t n_layers,
                         const uint32_t* masks, int32_t words, const int32_t* nodes, void* pool, size_t pool_bytes,
                         int32_t* lens_out, uint32_t* status_dev, hipStream_t stream) {
  uint8_t* first;
  kvtc_status st = check_call(cfg, batch, layer, n_layers, pool, pool_bytes, status_dev, &first);
  if (st == KVTC_OK) st = check_masks(*batch, masks, words);
  if (st != KVTC_OK) return st;
  if (misaligned(nodes, 4) || misaligned(lens_out, 4)) return KVTC_ERR_INVALID_ARG;
  if (batch->n_seqs == 0) return KVTC_OK;
  if (!nodes || !lens_out) return KVTC_ERR_INVALID_ARG;
  if (batch->n_seqs > kMaxGrid) return KVTC_ERR_UNSUPPORTED;
  // every workgroup of a sequence reads its length, rows, node, mask and pages
  const int64_t n = batch->n_seqs;
  if (overlap(lens_out, n, batch->kv_lens, n) || overlap(lens_out, n, batch->row_start, n + 1) ||
      overlap(lens_out, n, batch->page_table, n * batch->max_pages) || overlap(lens_out, n, nodes, n) ||
      overlap(lens_out, n, masks, (int64_t)batch->total_rows * words) ||
      overlap(lens_out, n, pool, cfg->layers * (layer_bytes(*cfg) / 4)))
    return KVTC_ERR_INVALID_ARG;
  MxKeepParams p{};
  p.b = *batch;
  p.H = cfg->kv_heads;
  p.n_layers = n_layers;
  p.pool_pages = cfg->pool_pages;
  p.words = words;
  p.pool = first;
  p.layer_bytes = layer_bytes(*cfg);
  p.masks = masks;
  p.nodes = nodes;
  p.lens_out = lens_out;
  p.status = status_dev;
  return launch_mx_keep(p, cfg->head_dim, cfg->bits_k, cfg->bits_v, stream) == hipSuccess ? KVTC_OK : KVTC_ERR_HIP;
}

}  // extern "C"
