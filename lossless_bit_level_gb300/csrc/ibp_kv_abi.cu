// C ABI of the 8-bit paged key/value cache: argument checks and launches (declared in
// include/ibp.h).
#include "ibp_kv.h"

namespace ibp {

namespace {

bool device_ptr(const void *p, size_t align) { return pointer_ok(p, Where::device_only, align); }
bool device_or_null(const void *p, size_t align) { return !p || device_ptr(p, align); }

bool float_dtype(int dtype) { return dtype == IBP_FP32 || dtype == IBP_FP16 || dtype == IBP_BF16; }

// Sizes only (no CUDA call).
int kv_geometry(const ibp_kv_cache *c) {
  if (!c) return IBP_ERR_ARG;
  if (c->code != IBP_KV_INT8 && c->code != IBP_KV_E4M3) return IBP_ERR_DTYPE;
  if (c->batch < 0 || c->n_heads <= 0 || c->n_pages < 0 || c->table_cols < 0 ||
      c->table_stride < c->table_cols)
    return IBP_ERR_ARG;
  if ((c->head_dim != 64 && c->head_dim != 128) ||
      (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 &&
       c->page_tokens != 128))
    return IBP_ERR_UNSUPPORTED;
  if (c->n_pages > 0x7FFFFFFF || c->n_heads > 4096 || c->batch > 65535 ||
      (int64_t)c->table_cols * c->page_tokens > KV_MAX_CAPACITY)
    return IBP_ERR_UNSUPPORTED;
  return IBP_OK;
}

bool kv_pointers(const ibp_kv_cache *c, bool with_lens = true) {
  return device_ptr(c->k_codes, 16) && device_ptr(c->v_codes, 16) && device_ptr(c->k_scales, 4) &&
         device_ptr(c->v_scales, 4) && device_ptr(c->d_table, 4) &&
         (!with_lens || device_ptr(c->d_lens, 4));
}

// A stride in elements: whole 16-byte pieces, so every head starts 16-byte aligned.
bool stride_ok(int64_t stride, int elem_bytes) {
  return stride >= 0 && stride <= (int64_t(1) << 40) && stride * elem_bytes % 16 == 0;
}

// Whether heads of `dim` elements, `heads` of them `head_stride` apart in each of n_rows rows
// `row_stride` apart, share an element (they are written by different threads).
bool heads_overlap(int64_t n_rows, int64_t row_stride, int64_t heads, int64_t head_stride, int64_t dim) {
  if ((n_rows > 1 && row_stride < dim) || (heads > 1 && head_stride < dim)) return true;
  if (n_rows <= 1 || heads <= 1) return false;
  if ((row_stride - dim) / head_stride >= heads - 1 || (head_stride - dim) / row_stride >= n_rows - 1)
    return false;  // whole rows, or whole columns of heads, one after another
  for (int64_t j = 1; j < heads; ++j) {  // head j against the rows around it
    const int64_t i = j * head_stride / row_stride, past = j * head_stride - i * row_stride;
    if ((i < n_rows && past < dim) || (i + 1 < n_rows && row_stride - past < dim)) return true;
  }
  return false;
}

bool ranges_overlap(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

}  // namespace

}  // namespace ibp

using namespace ibp;

extern "C" {

// What both appends ask of their rows; 1: there is nothing to do.
static int kv_append_check(const ibp_kv_cache *cache, const ibp_kv_rows *rows, int32_t *d_new_lens,
                           int32_t *d_status) {
  if (int rc = kv_geometry(cache)) return rc;
  if (!rows) return IBP_ERR_ARG;
  if (!float_dtype(rows->dtype)) return IBP_ERR_DTYPE;
  const int es = rows->dtype == IBP_FP32 ? 4 : 2;
  if (rows->n_rows < 0 || rows->n_rows > KV_MAX_CAPACITY || !stride_ok(rows->k_row_stride, es) ||
      !stride_ok(rows->k_head_stride, es) || !stride_ok(rows->v_row_stride, es) ||
      !stride_ok(rows->v_head_stride, es))
    return IBP_ERR_ARG;
  if (cache->batch == 0) return rows->n_rows == 0 ? 1 : IBP_ERR_ARG;
  if (!rows->d_cu && rows->n_rows % cache->batch != 0) return IBP_ERR_ARG;
  if (rows->n_rows == 0 && !d_new_lens) return 1;
  if (!kv_pointers(cache) || !device_or_null(rows->d_cu, 4) || !device_or_null(d_new_lens, 4) ||
      !device_or_null(d_status, 4) || d_new_lens == cache->d_lens)
    return IBP_ERR_ARG;
  if (rows->n_rows > 0 && (!device_ptr(rows->k, 16) || !device_ptr(rows->v, 16)))
    return IBP_ERR_ARG;
  return IBP_OK;
}

int ibp_kv_append(const ibp_kv_cache *cache, const ibp_kv_rows *rows, int32_t *d_new_lens,
                  int32_t *d_status, ibp_stream_t s) {
  if (int rc = kv_append_check(cache, rows, d_new_lens, d_status)) return rc > 0 ? IBP_OK : rc;
  return launch_kv_append(*cache, *rows, d_new_lens, d_status, reinterpret_cast<cudaStream_t>(s));
}

// Elements from the first of n rows of heads to past the last one (what no memory holds is held
// at 2^60).
static int64_t rows_span(int64_t n, int64_t row_stride, int64_t heads, int64_t head_stride, int64_t dim) {
  const int64_t most = int64_t(1) << 60;
  if (n <= 0) return 0;
  if (row_stride > 0 && n - 1 > most / row_stride) return most;
  return (n - 1) * row_stride + (heads - 1) * head_stride + dim;
}

// Rows of heads in memory that is read, or written.
struct HeadRows {
  const void *at;
  int64_t row_stride, head_stride, heads;
};

// Whether n rows of heads of `dim` elements that are written share an element with n rows that are
// read. Both may lie in one fused tensor, so that the stretches of memory that they span overlap
// while their elements do not: with one row stride it is the heads' places in a row that count.
// Rows of different strides in overlapping stretches are taken to share one.
static bool rows_overlap(const HeadRows &w, const HeadRows &r, int64_t n, int64_t dim, int elem_bytes) {
  const int64_t n_r = r.row_stride ? n : 1, heads_r = r.head_stride ? r.heads : 1;  // (broadcast: one of them)
  if (!ranges_overlap(w.at, (size_t)rows_span(n, w.row_stride, w.heads, w.head_stride, dim) * elem_bytes, r.at,
                      (size_t)rows_span(n_r, r.row_stride, heads_r, r.head_stride, dim) * elem_bytes))
    return false;
  if (n > 1 && n_r > 1 && w.row_stride != r.row_stride) return true;
  const int64_t far = int64_t(1) << 58, row = n > 1 ? w.row_stride : w.heads > 1 ? far - far % w.head_stride : far;
  const int64_t from = (reinterpret_cast<intptr_t>(r.at) - reinterpret_cast<intptr_t>(w.at)) / elem_bytes;
  // the common layouts, in a few steps: one's heads behind the other's within a row, or between them
  const int64_t in_row = from % row + (from % row < 0 ? row : 0);
  if (in_row >= rows_span(1, 0, w.heads, w.head_stride, dim) &&
      in_row + rows_span(1, 0, heads_r, r.head_stride, dim) <= row)
    return false;
  if (w.heads > 1 && (heads_r == 1 || w.head_stride == r.head_stride) && row % w.head_stride == 0) {
    const int64_t in_head = in_row % w.head_stride;
    if (in_head >= dim && in_head + dim <= w.head_stride) return false;
  }
  // every head read against every head written, in the rows around it: those k rows on, of which
  // there are n - 1 forwards and n_r - 1 back
  for (int64_t i = 0; i < heads_r; ++i)
    for (int64_t j = 0; j < w.heads; ++j) {
      const int64_t apart = from + i * r.head_stride - j * w.head_stride, below = apart / row - (apart % row < 0);
      for (int64_t k = below; k <= below + 1; ++k) {
        const int64_t held = k < 1 - n_r ? 1 - n_r : k > n - 1 ? n - 1 : k, past = apart - held * row;
        if (past < dim && -past < dim) return true;
      }
    }
  return false;
}

int ibp_kv_append_rotated(const ibp_kv_cache *cache, const ibp_kv_rows *rows,
                          const ibp_kv_rotation *rotation, const ibp_kv_turned *queries,
                          int32_t *d_new_lens, int32_t *d_status, ibp_stream_t s) {
  if (!rotation) return IBP_ERR_ARG;
  if (int rc = kv_geometry(cache)) return rc;
  const ibp_kv_rotation &t = *rotation;
  if (t.dim < 16 || t.dim > cache->head_dim || t.dim % 16 != 0 || t.axes < 1 || t.axes > 4 ||
      t.n_positions < 1 || t.n_positions > KV_MAX_CAPACITY)
    return IBP_ERR_ARG;
  for (int i = 0; i < t.dim / 2; ++i)
    if (t.axis[i] >= t.axes) return IBP_ERR_ARG;
  const int nothing = kv_append_check(cache, rows, d_new_lens, d_status);
  if (nothing < 0) return nothing;
  const int es = rows->dtype == IBP_FP32 ? 4 : 2;
  if (queries) {
    const ibp_kv_turned &q = *queries;
    if (q.q_heads < 1 || q.q_heads > 65535 || !stride_ok(q.q_row_stride, es) ||
        !stride_ok(q.q_head_stride, es) || !stride_ok(q.out_row_stride, es) ||
        !stride_ok(q.out_head_stride, es) ||
        heads_overlap(rows->n_rows, q.out_row_stride, q.q_heads, q.out_head_stride, cache->head_dim))
      return IBP_ERR_ARG;
  }
  if (nothing) return IBP_OK;
  if (!device_ptr(t.d_table, 16) || !device_or_null(t.d_positions, 4)) return IBP_ERR_ARG;
  if (queries && rows->n_rows > 0) {
    const ibp_kv_turned &q = *queries;
    if (!device_ptr(q.q, 16) || !device_ptr(q.out, 16)) return IBP_ERR_ARG;
    const bool same = q.q == q.out && q.q_row_stride == q.out_row_stride && q.q_head_stride == q.out_head_stride;
    const HeadRows out = {q.out, q.out_row_stride, q.out_head_stride, q.q_heads};
    // queries are written while rows are still read
    const HeadRows from = {q.q, q.q_row_stride, q.q_head_stride, q.q_heads};
    const HeadRows k = {rows->k, rows->k_row_stride, rows->k_head_stride, cache->n_heads};
    const HeadRows v = {rows->v, rows->v_row_stride, rows->v_head_stride, cache->n_heads};
    if ((!same && rows_overlap(out, from, rows->n_rows, cache->head_dim, es)) ||
        rows_overlap(out, k, rows->n_rows, cache->head_dim, es) ||
        rows_overlap(out, v, rows->n_rows, cache->head_dim, es))
      return IBP_ERR_ARG;
  }
  return launch_kv_append_rotated(*cache, *rows, t, queries, d_new_lens, d_status,
                                  reinterpret_cast<cudaStream_t>(s));
}

int ibp_kv_read(const ibp_kv_cache *cache, const int32_t *d_begin, int64_t n_out, void *k_out,
                void *v_out, int dtype, int32_t *d_status, ibp_stream_t s) {
  if (int rc = kv_geometry(cache)) return rc;
  if (!float_dtype(dtype)) return IBP_ERR_DTYPE;
  if (n_out < 0 || n_out > KV_MAX_CAPACITY) return IBP_ERR_ARG;
  if (n_out == 0 || cache->batch == 0 || (!k_out && !v_out)) return IBP_OK;
  if (!kv_pointers(cache) || !device_or_null(d_begin, 4) || !device_or_null(k_out, 16) ||
      !device_or_null(v_out, 16) || !device_or_null(d_status, 4))
    return IBP_ERR_ARG;
  return launch_kv_read(*cache, d_begin, n_out, k_out, v_out, dtype, d_status,
                        reinterpret_cast<cudaStream_t>(s));
}

static int kv_query_sizes(const ibp_kv_cache *cache, int64_t n_rows, int64_t max_q,
                          int32_t q_heads) {
  if (int rc = kv_geometry(cache)) return rc;
  if (n_rows < 0 || max_q < 0 || n_rows > KV_MAX_CAPACITY || max_q > KV_MAX_CAPACITY ||
      q_heads <= 0 || q_heads % cache->n_heads != 0 || q_heads > 65535)
    return IBP_ERR_ARG;
  // the rows of a K/V head of one sequence are counted in 32 bits
  if (n_rows * (q_heads / cache->n_heads) > KV_MAX_CAPACITY) return IBP_ERR_UNSUPPORTED;
  return IBP_OK;
}

int ibp_kv_attention_scratch_bytes(const ibp_kv_cache *cache, int64_t n_rows, int64_t max_q,
                                   int32_t q_heads, int with_weights, size_t *bytes) {
  if (!bytes) return IBP_ERR_ARG;
  if (int rc = kv_query_sizes(cache, n_rows, max_q, q_heads)) return rc;
  *bytes = kv_attention_scratch_bytes(*cache, n_rows, max_q, q_heads, with_weights != 0);
  return IBP_OK;
}

// Query rows as every call takes them (no CUDA call).
static int kv_query_rows(const ibp_kv_cache *cache, const ibp_kv_query *query) {
  if (!query) return IBP_ERR_ARG;
  if (int rc = kv_query_sizes(cache, query->n_rows, query->max_q, query->q_heads)) return rc;
  const ibp_kv_query &q = *query;
  if (q.dtype != IBP_FP16 && q.dtype != IBP_BF16) return IBP_ERR_DTYPE;
  if (!stride_ok(q.q_row_stride, 2) || !stride_ok(q.q_head_stride, 2)) return IBP_ERR_ARG;
  if (!q.d_cu && q.n_rows != cache->batch * q.max_q) return IBP_ERR_ARG;
  if (q.n_rows > 0 && q.max_q == 0) return IBP_ERR_ARG;
  return IBP_OK;
}

// And where attention writes for them.
static int kv_query_out(const ibp_kv_cache *cache, const ibp_kv_query &q) {
  if (!stride_ok(q.out_row_stride, 2) || !stride_ok(q.out_head_stride, 2) ||
      heads_overlap(q.n_rows, q.out_row_stride, q.q_heads, q.out_head_stride, cache->head_dim) ||
      !(q.scale == q.scale))
    return IBP_ERR_ARG;
  return IBP_OK;
}

int ibp_kv_attention(const ibp_kv_cache *cache, const ibp_kv_query *query, void *d_scratch,
                     size_t scratch_bytes, int32_t *d_status, ibp_stream_t s) {
  if (int rc = kv_query_rows(cache, query)) return rc;
  const ibp_kv_query &q = *query;
  if (int rc = kv_query_out(cache, q)) return rc;
  if (q.d_weights && !(q.decay == q.decay)) return IBP_ERR_ARG;
  if (q.d_weights_in && !q.d_weights) return IBP_ERR_ARG;
  if (q.d_weights && q.weights_stride < 0) return IBP_ERR_ARG;
  if (cache->batch == 0 || (q.n_rows == 0 && !q.d_weights)) return IBP_OK;
  if (q.d_weights &&
      q.weights_stride < (int64_t)cache->table_cols * cache->page_tokens)
    return IBP_ERR_ARG;
  if (scratch_bytes <
      kv_attention_scratch_bytes(*cache, q.n_rows, q.max_q, q.q_heads, q.d_weights != nullptr))
    return IBP_ERR_ARG;
  if (!kv_pointers(cache) || !device_ptr(d_scratch, 16) || !device_or_null(q.d_lse, 4) ||
      !device_or_null(q.d_cu, 4) || !device_or_null(q.d_weights_in, 4) ||
      !device_or_null(q.d_weights, 4) || !device_or_null(d_status, 4))
    return IBP_ERR_ARG;
  if (q.n_rows > 0 && (!device_ptr(q.q, 16) || !device_ptr(q.out, 16))) return IBP_ERR_ARG;
  return launch_kv_attention(*cache, q, d_scratch, d_status, reinterpret_cast<cudaStream_t>(s));
}

int ibp_kv_bounds(const ibp_kv_cache *cache, int8_t *d_bounds, const int32_t *d_begin,
                  int32_t *d_status, ibp_stream_t s) {
  if (int rc = kv_geometry(cache)) return rc;
  if (cache->batch == 0) return IBP_OK;
  if (!kv_pointers(cache) || !device_ptr(d_bounds, 16) || !device_or_null(d_begin, 4) ||
      !device_or_null(d_status, 4))
    return IBP_ERR_ARG;
  return launch_kv_bounds(*cache, d_bounds, d_begin, d_status, reinterpret_cast<cudaStream_t>(s));
}

// Whether lists of `pages` hold a sequence's first page and those of its rows.
static int kv_pages_ok(const ibp_kv_cache *cache, int64_t n_rows, int64_t max_q, int64_t pages) {
  const int64_t most = max_q < n_rows ? max_q : n_rows, P = cache->page_tokens;
  const int64_t own = most > 0 ? (most - 1 + P - 1) / P + 1 : 0;
  if (pages < own + 1 || pages > KV_MAX_CAPACITY / P) return IBP_ERR_ARG;
  return IBP_OK;
}

int ibp_kv_select_scratch_bytes(const ibp_kv_cache *cache, size_t *bytes) {
  if (!bytes) return IBP_ERR_ARG;
  if (int rc = kv_geometry(cache)) return rc;
  *bytes = kv_select_scratch_bytes(*cache);
  return IBP_OK;
}

int ibp_kv_select(const ibp_kv_cache *cache, const int8_t *d_bounds, const ibp_kv_query *query,
                  int64_t pages, int32_t *d_columns, void *d_scratch, size_t scratch_bytes,
                  int32_t *d_status, ibp_stream_t s) {
  if (int rc = kv_query_rows(cache, query)) return rc;
  const ibp_kv_query &q = *query;
  if (int rc = kv_pages_ok(cache, q.n_rows, q.max_q, pages)) return rc;
  if (scratch_bytes < kv_select_scratch_bytes(*cache)) return IBP_ERR_ARG;
  if (cache->batch == 0) return IBP_OK;
  if (!kv_pointers(cache) || !device_ptr(d_bounds, 16) || !device_ptr(d_columns, 4) ||
      !device_or_null(q.d_cu, 4) || !device_ptr(d_scratch, 16) || !device_or_null(d_status, 4))
    return IBP_ERR_ARG;
  if (q.n_rows > 0 && !device_ptr(q.q, 16)) return IBP_ERR_ARG;
  return launch_kv_select(*cache, d_bounds, q, pages, d_columns, d_scratch, d_status,
                          reinterpret_cast<cudaStream_t>(s));
}

int ibp_kv_attention_selected_scratch_bytes(const ibp_kv_cache *cache, int64_t n_rows, int64_t max_q,
                                            int32_t q_heads, int64_t pages, size_t *bytes) {
  if (!bytes) return IBP_ERR_ARG;
  if (int rc = kv_query_sizes(cache, n_rows, max_q, q_heads)) return rc;
  if (int rc = kv_pages_ok(cache, n_rows, max_q, pages)) return rc;
  *bytes = kv_selected_scratch_bytes(*cache, n_rows, max_q, q_heads);
  return IBP_OK;
}

int ibp_kv_attention_selected(const ibp_kv_cache *cache, const ibp_kv_query *query,
                              const int32_t *d_columns, int64_t pages, void *d_scratch,
                              size_t scratch_bytes, int32_t *d_status, ibp_stream_t s) {
  if (int rc = kv_query_rows(cache, query)) return rc;
  const ibp_kv_query &q = *query;
  if (int rc = kv_query_out(cache, q)) return rc;
  if (q.d_weights || q.d_weights_in) return IBP_ERR_ARG;
  if (int rc = kv_pages_ok(cache, q.n_rows, q.max_q, pages)) return rc;
  if (cache->batch == 0 || q.n_rows == 0) return IBP_OK;
  if (scratch_bytes < kv_selected_scratch_bytes(*cache, q.n_rows, q.max_q, q.q_heads)) return IBP_ERR_ARG;
  if (!kv_pointers(cache) || !device_ptr(d_scratch, 16) || !device_or_null(q.d_lse, 4) ||
      !device_or_null(q.d_cu, 4) || !device_ptr(d_columns, 4) || !device_or_null(d_status, 4) ||
      !device_ptr(q.q, 16) || !device_ptr(q.out, 16))
    return IBP_ERR_ARG;
  return launch_kv_attention_selected(*cache, q, d_columns, pages, d_scratch, d_status,
                                      reinterpret_cast<cudaStream_t>(s));
}

static int kv_groups_ok(const ibp_kv_cache *cache, int64_t n_groups, int64_t group_rows) {
  return n_groups < 0 || n_groups > cache->batch || group_rows < 0 || group_rows > KV_MAX_CAPACITY
             ? IBP_ERR_ARG
             : IBP_OK;
}

int ibp_kv_attention_shared_scratch_bytes(const ibp_kv_cache *cache, int64_t n_rows, int64_t max_q,
                                          int32_t q_heads, int64_t n_groups, int64_t group_rows,
                                          size_t *bytes) {
  if (!bytes) return IBP_ERR_ARG;
  if (int rc = kv_query_sizes(cache, n_rows, max_q, q_heads)) return rc;
  if (int rc = kv_groups_ok(cache, n_groups, group_rows)) return rc;
  *bytes = kv_shared_scratch_bytes(*cache, n_rows, max_q, q_heads, n_groups, group_rows);
  return IBP_OK;
}

int ibp_kv_attention_shared(const ibp_kv_cache *cache, const ibp_kv_query *query, const int32_t *d_groups,
                            const int32_t *d_prefix, int64_t n_groups, int64_t group_rows,
                            void *d_scratch, size_t scratch_bytes, int32_t *d_status, ibp_stream_t s) {
  if (int rc = kv_query_rows(cache, query)) return rc;
  const ibp_kv_query &q = *query;
  if (int rc = kv_query_out(cache, q)) return rc;
  if (int rc = kv_groups_ok(cache, n_groups, group_rows)) return rc;
  if (q.d_weights || q.d_weights_in) return IBP_ERR_ARG;
  if (cache->batch == 0 || q.n_rows == 0) return IBP_OK;
  if (scratch_bytes < kv_shared_scratch_bytes(*cache, q.n_rows, q.max_q, q.q_heads, n_groups, group_rows))
    return IBP_ERR_ARG;
  if (!kv_pointers(cache) || !device_ptr(d_scratch, 16) || !device_or_null(q.d_lse, 4) ||
      !device_or_null(q.d_cu, 4) || !device_or_null(d_status, 4) || !device_ptr(q.q, 16) ||
      !device_ptr(q.out, 16) || (n_groups > 0 && (!device_ptr(d_groups, 4) || !device_ptr(d_prefix, 4))))
    return IBP_ERR_ARG;
  return launch_kv_attention_shared(*cache, q, d_groups, d_prefix, n_groups, group_rows, d_scratch, d_status,
                                    reinterpret_cast<cudaStream_t>(s));
}

int ibp_kv_evict_scratch_bytes(const ibp_kv_cache *cache, int64_t budget, size_t *bytes) {
  if (!bytes) return IBP_ERR_ARG;
  if (int rc = kv_geometry(cache)) return rc;
  if (budget < 1 || budget > KV_MAX_CAPACITY) return IBP_ERR_ARG;
  *bytes = kv_evict_scratch_bytes(*cache, budget);
  return IBP_OK;
}

int ibp_kv_evict(const ibp_kv_cache *cache, const float *d_weights, int64_t weights_stride,
                 int64_t budget, int64_t recent, const ibp_kv_cache *dst, int32_t *d_new_lens,
                 float *d_new_weights, int64_t new_weights_stride, int32_t *d_kept,
                 void *d_scratch, size_t scratch_bytes, int32_t *d_status, ibp_stream_t s) {
  if (int rc = kv_geometry(cache)) return rc;
  if (int rc = kv_geometry(dst)) return rc;
  const int64_t cap = (int64_t)cache->table_cols * cache->page_tokens;
  if (budget < 1 || budget > KV_MAX_CAPACITY || recent < 0 || recent > budget ||
      weights_stride < cap || (d_new_weights && new_weights_stride < budget))
    return IBP_ERR_ARG;
  if (dst->batch != cache->batch || dst->n_heads != cache->n_heads ||
      dst->page_tokens != cache->page_tokens || dst->head_dim != cache->head_dim ||
      dst->code != cache->code ||
      (int64_t)dst->table_cols * dst->page_tokens < (budget < cap ? budget : cap))
    return IBP_ERR_ARG;
  if (cache->batch == 0) return IBP_OK;
  if (scratch_bytes < kv_evict_scratch_bytes(*cache, budget)) return IBP_ERR_ARG;
  if (!kv_pointers(cache) || !kv_pointers(dst, false) || !device_ptr(d_weights, 4) ||
      !device_ptr(d_new_lens, 4) || !device_or_null(d_new_weights, 4) ||
      !device_or_null(d_kept, 4) || !device_ptr(d_scratch, 16) || !device_or_null(d_status, 4) ||
      d_new_lens == cache->d_lens)
    return IBP_ERR_ARG;
  const size_t lists = (size_t)cache->batch * cache->n_heads * sizeof(float);
  if (d_new_weights &&
      ranges_overlap(d_weights, lists * weights_stride, d_new_weights, lists * new_weights_stride))
    return IBP_ERR_ARG;
  return launch_kv_evict(*cache, d_weights, weights_stride, budget, recent, *dst, d_new_lens,
                         d_new_weights, new_weights_stride, d_kept, d_scratch, d_status,
                         reinterpret_cast<cudaStream_t>(s));
}

}  // extern "C"
