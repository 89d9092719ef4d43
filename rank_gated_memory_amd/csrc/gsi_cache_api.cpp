// Entry points of the paged key-value cache: argument checks.
#include "gsi_cache.h"

namespace gsi {
namespace {

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int size_of(int dtype) { return dtype == GSI_FP32 ? 4 : 2; }

// A stride in elements over `n` things: `n` of them, in bytes and beside two
// others, stay within 64 bits.
inline bool stride_ok(int64_t stride, int64_t n, int d) { return stride >= d && stride <= (INT64_MAX >> 5) / n; }

gsi_status check_cache(const gsi_cache *c) {
  if (!c) return GSI_E_NULL;
  if (c->dtype != GSI_FP32 && c->dtype != GSI_BF16) return GSI_E_DTYPE;
  if (c->pages < 1 || c->page < 8 || c->page > 4096 || (c->page & (c->page - 1)) || c->heads < 1 || c->heads > 1024 ||
      c->d < 8 || c->d > 256 || c->d % 8)
    return GSI_E_SHAPE;
  if (!stride_ok(c->page_stride, c->pages, c->d) || !stride_ok(c->head_stride, c->heads, c->d) ||
      !stride_ok(c->slot_stride, c->page, c->d) || c->slot_stride >= (1 << 24))
    return GSI_E_SHAPE;
  if (!c->K || !c->V) return GSI_E_NULL;
  const int vec = 16 / size_of(c->dtype);
  if (!aligned(c->K, 16) || !aligned(c->V, 16) || c->page_stride % vec || c->head_stride % vec ||
      c->slot_stride % vec || !aligned(c->mass, 4) || !aligned(c->age, 4))
    return GSI_E_ALIGN;
  return GSI_OK;
}

gsi_status check_table(const gsi_table *t, int page) {
  if (!t) return GSI_E_NULL;
  if (t->S < 0 || t->S >= (1 << 24) || t->most < 0 || (int64_t)t->most * page > (1 << 30) || t->ld < t->most ||
      t->ld > INT64_MAX / 8 / (t->S + 1))
    return GSI_E_SHAPE;
  if (!t->table && t->S > 0 && t->most > 0) return GSI_E_NULL;
  return aligned(t->table, 4) ? GSI_OK : GSI_E_ALIGN;
}

gsi_status check_heads(const gsi_heads *h, int32_t rows, int d, int dtype) {
  if (!h) return GSI_E_NULL;
  if (h->n < 1 || h->n > 4096) return GSI_E_SHAPE;
  const bool many_rows = rows > 1, many_heads = h->n > 1;
  if ((many_rows && !stride_ok(h->row, rows, d)) || (many_heads && !stride_ok(h->head, h->n, d))) return GSI_E_SHAPE;
  if (!h->p && rows > 0) return GSI_E_NULL;
  const int vec = 16 / size_of(dtype);
  return aligned(h->p, 16) && (!many_rows || h->row % vec == 0) && (!many_heads || h->head % vec == 0) ? GSI_OK
                                                                                                       : GSI_E_ALIGN;
}

gsi_status check_rotation(const gsi_rotation *r, int d) {
  if (!r) return GSI_E_NULL;
  if (r->layout != GSI_ROTARY_PAIRS && r->layout != GSI_ROTARY_HALVES) return GSI_E_ARG;
  if (r->d < 2 || r->d % 2 || r->start < 0 || r->d > d || r->start > d - r->d) return GSI_E_SHAPE;
  if (!r->freq) return GSI_E_NULL;
  return aligned(r->freq, 8) ? GSI_OK : GSI_E_ALIGN;
}

gsi_status check_positions(const void *positions, int pos_bytes) {
  if (pos_bytes != 4 && pos_bytes != 8) return GSI_E_DTYPE;
  return aligned(positions, pos_bytes) ? GSI_OK : GSI_E_ALIGN;
}

Rows rows_of(const gsi_heads *h, int32_t rows, int dtype) {
  if (!h) return {};
  const int es = size_of(dtype);
  return {static_cast<uint8_t *>(h->p), rows > 1 ? h->row * es : 0, h->n > 1 ? h->head * es : 0, h->n};
}

Pool pool_of(const gsi_cache *c, const gsi_table *t) {
  const int es = size_of(c->dtype);
  Pool p{};
  p.K = static_cast<uint8_t *>(c->K);
  p.V = static_cast<uint8_t *>(c->V);
  p.mass = c->mass;
  p.age = c->age;
  p.table = t->table;
  p.page_stride = c->page_stride * es;
  p.head_stride = c->head_stride * es;
  p.slot_stride = c->slot_stride * es;
  p.ld = t->ld;
  p.pages = c->pages;
  p.shift = __builtin_ctz((unsigned)c->page);
  p.heads = c->heads;
  p.d = c->d;
  p.S = t->S;
  p.most = t->most;
  return p;
}

}  // namespace
}  // namespace gsi

using namespace gsi;

#define GSI_CHECK(call)            \
  do {                             \
    const gsi_status s_ = (call);  \
    if (s_ != GSI_OK) return s_;   \
  } while (0)

extern "C" {

gsi_status gsi_rotary(const gsi_rotation *r, const gsi_heads *x, const gsi_heads *y, int32_t T,
                      int32_t d, int32_t dtype, const void *positions, int32_t pos_bytes,
                      void *stream) {
  if (dtype != GSI_FP32 && dtype != GSI_BF16) return GSI_E_DTYPE;
  if (T < 0 || d < 8 || d > 256 || d % 8) return GSI_E_SHAPE;
  GSI_CHECK(check_rotation(r, d));
  GSI_CHECK(check_heads(x, T, d, dtype));
  GSI_CHECK(check_heads(y, T, d, dtype));
  if (x->n != y->n) return GSI_E_SHAPE;
  GSI_CHECK(check_positions(positions, pos_bytes));
  if (T == 0) return GSI_OK;
  if (!positions) return GSI_E_NULL;
  RotateArgs a{};
  a.q = rows_of(x, T, dtype);
  a.qo = rows_of(y, T, dtype);
  a.freq = r->freq;
  a.positions = positions;
  a.amplitude = r->amplitude;
  a.pos_bytes = pos_bytes;
  a.T = T;
  a.d = d;
  a.turned = r->d;
  a.start = r->start;
  return launch_rotate(a, dtype, r->layout, static_cast<hipStream_t>(stream));
}

gsi_status gsi_cache_append(const gsi_cache *cache, const gsi_table *table, const int32_t *seq,
                            const int32_t *slots, const gsi_heads *k, const gsi_heads *v, int32_t T,
                            const gsi_rotation *r, const void *positions, int32_t pos_bytes,
                            const gsi_heads *q, const gsi_heads *q_out, void *stream) {
  GSI_CHECK(check_cache(cache));
  GSI_CHECK(check_table(table, cache->page));
  if (T < 0) return GSI_E_SHAPE;
  const int d = cache->d, dtype = cache->dtype;
  GSI_CHECK(check_heads(k, T, d, dtype));
  GSI_CHECK(check_heads(v, T, d, dtype));
  if (k->n != cache->heads || v->n != cache->heads) return GSI_E_SHAPE;
  if (r) GSI_CHECK(check_rotation(r, d));
  if (!q != !q_out) return GSI_E_NULL;
  if (q) {
    GSI_CHECK(check_heads(q, T, d, dtype));
    GSI_CHECK(check_heads(q_out, T, d, dtype));
    if (q->n != q_out->n) return GSI_E_SHAPE;
  }
  if (positions || r) GSI_CHECK(check_positions(positions, pos_bytes));
  if (!aligned(seq, 4) || !aligned(slots, 4)) return GSI_E_ALIGN;
  if (T == 0) return GSI_OK;
  if (!slots || (r && !positions)) return GSI_E_NULL;
  RotateArgs a{};
  a.q = rows_of(q, T, dtype);
  a.qo = rows_of(q_out, T, dtype);
  a.k = rows_of(k, T, dtype);
  a.v = rows_of(v, T, dtype);
  a.c = pool_of(cache, table);
  a.seq = seq;
  a.slots = slots;
  a.freq = r ? r->freq : nullptr;
  a.positions = positions;
  a.amplitude = r ? r->amplitude : 1.f;
  a.pos_bytes = pos_bytes;
  a.T = T;
  a.d = d;
  a.turned = r ? r->d : 0;
  a.start = r ? r->start : 0;
  return launch_rotate(a, dtype, r ? r->layout : GSI_ROTARY_PAIRS, static_cast<hipStream_t>(stream));
}

size_t gsi_cache_attend_workspace(const gsi_cache *cache, const gsi_table *table, int32_t q_heads,
                                  int32_t accumulate) {
  if (check_cache(cache) != GSI_OK || check_table(table, cache->page) != GSI_OK) return 0;
  if (q_heads < 1 || q_heads > 4096 || q_heads % cache->heads) return 0;
  const Pool pool = pool_of(cache, table);
  return attend_counts(pool) ? attend_workspace(pool, cache->dtype, q_heads, accumulate != 0) : 0;
}

gsi_status gsi_cache_attend(const gsi_cache *cache, const gsi_table *table, const int32_t *lengths,
                            const gsi_heads *q, const gsi_heads *out, float scale, int32_t window,
                            int32_t accumulate, float *lse, void *ws, size_t ws_bytes,
                            void *stream) {
  GSI_CHECK(check_cache(cache));
  GSI_CHECK(check_table(table, cache->page));
  const int32_t S = table->S;
  GSI_CHECK(check_heads(q, S, cache->d, cache->dtype));
  GSI_CHECK(check_heads(out, S, cache->d, cache->dtype));
  if (q->n != out->n || q->n % cache->heads || window < 0) return GSI_E_SHAPE;
  if (accumulate && !cache->mass) return GSI_E_NULL;
  if (!aligned(lengths, 4) || !aligned(lse, 4) || !aligned(ws, 16)) return GSI_E_ALIGN;
  if (S == 0) return GSI_OK;
  if (!lengths) return GSI_E_NULL;
  AttendArgs a{};
  a.c = pool_of(cache, table);
  if (!attend_counts(a.c)) return GSI_E_SHAPE;
  const size_t need = attend_workspace(a.c, cache->dtype, q->n, accumulate != 0);
  if (need > 0 && !ws) return GSI_E_NULL;
  if (ws_bytes < need) return GSI_E_WORKSPACE;
  a.q = rows_of(q, S, cache->dtype);
  a.out = rows_of(out, S, cache->dtype);
  a.lengths = lengths;
  a.lse = lse;
  a.ws = static_cast<uint8_t *>(ws);
  a.scale = scale;
  a.window = window;
  a.group = q->n / cache->heads;
  a.accumulate = accumulate != 0;
  return launch_attend(a, cache->dtype, static_cast<hipStream_t>(stream));
}

gsi_status gsi_cache_evict(const gsi_cache *cache, const gsi_table *table, const int32_t *lengths,
                           int32_t budget, int32_t recent, const gsi_table *to,
                           int32_t *lengths_out, int32_t *from, void *stream) {
  GSI_CHECK(check_cache(cache));
  GSI_CHECK(check_table(table, cache->page));
  if (budget < 1 || budget > (1 << 20) || recent < 0 || recent > budget ||
      (int64_t)table->most * cache->page > (1 << 19))
    return GSI_E_SHAPE;
  if (to) {
    GSI_CHECK(check_table(to, cache->page));
    if (to->S != table->S || (int64_t)to->most * cache->page < budget) return GSI_E_SHAPE;
  }
  if (!aligned(lengths, 4) || !aligned(lengths_out, 4) || !aligned(from, 4)) return GSI_E_ALIGN;
  if (table->S == 0) return GSI_OK;
  if (!cache->mass || !lengths || !from) return GSI_E_NULL;
  if (lengths_out == lengths) return GSI_E_ARG;
  EvictArgs a{};
  a.c = pool_of(cache, table);
  if (to) {
    a.to = to->table;
    a.to_ld = to->ld;
  }
  a.lengths = lengths;
  a.lengths_out = lengths_out;
  a.from = from;
  a.budget = budget;
  a.recent = recent;
  return launch_evict(a, cache->dtype, static_cast<hipStream_t>(stream));
}

}  // extern "C"
