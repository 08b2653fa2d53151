// Shared by the kernels that append rows to the 8-bit paged key/value cache: which page a
// work item is for, and the rounding of values and of the codes that are there already.
#pragma once

#include "ibp_kv_device.cuh"

namespace ibp {

namespace {

__host__ __device__ constexpr int page_shift(int page_tokens) {
  return page_tokens == 16 ? 4 : page_tokens == 32 ? 5 : page_tokens == 64 ? 6 : 7;
}

// Work item -> (sequence, page): sequence b's items start at cu[b]/P + 2b (its rows
// touch at most (rows - 1)/P + 2 pages, so items of two sequences never overlap).
struct AppendPlace {
  int64_t lo, t0, end;  // first row of the sequence; tokens t0 .. end - 1 of the page and past it
  int b, len, page;     // page < 0: nothing to do
};

// Page sizes: a constant of the kernel, or known at launch. (Where it is a constant, shifts in place
// of the divisions cost an append of 8 x 4,096 tokens 147.3 -> 148.9 us.)
template <int P>
struct FixedPage {
  template <typename T>
  __device__ __forceinline__ T of(T tokens) const { return tokens / P; }
  __device__ __forceinline__ int64_t start(int64_t page) const { return page * P; }
};
struct ShiftedPage {
  int shift;
  template <typename T>
  __device__ __forceinline__ T of(T tokens) const { return tokens >> shift; }
  __device__ __forceinline__ int64_t start(int64_t page) const { return page << shift; }
};

template <typename Page>
__device__ __forceinline__ int64_t first_item(const ibp_kv_rows &r, int b, Page page) {
  return page.of(max(__ldg(r.d_cu + b), 0)) + 2 * (int64_t)b;
}

template <typename Page>
__device__ __forceinline__ AppendPlace place_of(const ibp_kv_cache &c, const ibp_kv_rows &r,
                                                int64_t each, int b, int64_t nth, Page page,
                                                bool reports, int32_t *new_lens,
                                                int32_t *status) {
  AppendPlace p;
  p.b = b;
  p.page = -1;
  int64_t hi;
  kv_row_range(r.d_cu, r.n_rows, each, b, status, &p.lo, &hi);
  p.len = kv_len(c, b, status);
  const int64_t cap = page.start(c.table_cols);
  const int64_t all = p.len + (hi - p.lo);
  p.end = all < cap ? all : cap;
  if (nth < 0) return p;
  if (nth == 0 && reports) {
    if (p.end != all) report(status, IBP_ERR_INDEX);
    if (new_lens) new_lens[b] = (int32_t)p.end;
  }
  p.t0 = page.start(page.of(p.len) + nth);
  if (p.t0 < p.end && hi > p.lo) p.page = kv_page(c, b, (int)page.of(p.t0), status);
  return p;
}

// 16 values times the inverse scale to 16 codes; ANY: some may be infinite, NaN or past
// what the scale covers.
template <int DT, int CODE, bool ANY>
__device__ __forceinline__ uint4 encode16(const Raw16<DT> &x, float inverse) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[4];
    x.four(i, y);
    mul4(y, inverse);
    w[i] = ANY ? kv_encode4_any<CODE>(y[0], y[1], y[2], y[3])
               : kv_encode4<CODE>(y[0], y[1], y[2], y[3]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of tokens that were there, moved to a larger scale.
template <int CODE>
__device__ __forceinline__ uint4 rescale16(uint4 old, float ratio) {
  const uint32_t o[4] = {old.x, old.y, old.z, old.w};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y[4];
    kv_decode4<CODE>(o[i], y);
    mul4(y, ratio);
    w[i] = kv_encode4<CODE>(y[0], y[1], y[2], y[3]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DT>
__device__ __noinline__ float largest_finite(const Raw16<DT> &x, float most) {
  for (int i = 0; i < 4; ++i) {
    float y[4];
    x.four(i, y);
    for (int k = 0; k < 4; ++k) most = fmaxf(most, finite_abs(y[k]));
  }
  return most;
}

}  // namespace

}  // namespace ibp
