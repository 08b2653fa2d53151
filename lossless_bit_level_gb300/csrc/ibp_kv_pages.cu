// Append and read of the 8-bit paged key/value cache (declared in include/ibp.h).
#include "ibp_kv_device.cuh"

namespace ibp {

namespace {

// scale = max |x| / qmax over a page's tile, code = rn(x / scale): bound by HBM, 3 bytes
// moved an element (bf16) for about two operations. One CTA quantises what one (page, head)
// tile of K or V receives: its source comes in 16-byte loads and its codes leave in 16-byte
// stores, and the values stay in registers as they came between the maximum (of the
// magnitude bits, two 16-bit elements at a time) and the rounding, so rows are read once
// and codes written once. A tile a CTA needs no exchange between CTAs for the scale.
// 8 prompts of 4,096 tokens, 32 heads of 128 bf16 (805 MB moved): 149 us, 5.4 TB/s.

// Work item -> (sequence, page): sequence b's items start at cu[b]/P + 2b (its rows
// touch at most (rows - 1)/P + 2 pages, so items of two sequences never overlap).
struct AppendPlace {
  int64_t lo, t0, end;  // first row of the sequence; tokens t0 .. end - 1 of the page and past it
  int b, len, page;     // page < 0: nothing to do
};

template <int P>
__device__ __forceinline__ int64_t first_item(const ibp_kv_rows &r, int b) {
  return max(__ldg(r.d_cu + b), 0) / P + 2 * (int64_t)b;
}

template <int P>
__device__ __forceinline__ AppendPlace place_of(const ibp_kv_cache &c, const ibp_kv_rows &r,
                                                int64_t each, int b, int64_t nth, bool reports,
                                                int32_t *new_lens, int32_t *status) {
  AppendPlace p;
  p.b = b;
  p.page = -1;
  int64_t hi;
  kv_row_range(r.d_cu, r.n_rows, each, b, status, &p.lo, &hi);
  p.len = kv_len(c, b, status);
  const int64_t cap = (int64_t)c.table_cols * P;
  const int64_t all = p.len + (hi - p.lo);
  p.end = all < cap ? all : cap;
  if (nth < 0) return p;
  if (nth == 0 && reports) {
    if (p.end != all) report(status, IBP_ERR_INDEX);
    if (new_lens) new_lens[b] = (int32_t)p.end;
  }
  p.t0 = (p.len / P + nth) * P;
  if (p.t0 < p.end && hi > p.lo) p.page = kv_page(c, b, (int)(p.t0 / P), status);
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

template <int P, int D, int DT, int CODE>
__global__ void __launch_bounds__(Tile<P, D>::threads)
    kv_append_kernel(ibp_kv_cache c, ibp_kv_rows r, int64_t each, int64_t items_each,
                     int32_t *new_lens, int32_t *status) {
  constexpr int T = Tile<P, D>::threads, G = Tile<P, D>::per_thread, GD = D / 16;
  __shared__ uint32_t sm[32];
  const int64_t item = blockIdx.x;
  const int head = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  int b;
  int64_t nth;
  if (r.d_cu) {
    // starts rise with b: the last one that is not past the item
    int below = 0;
    for (int k0 = 0; k0 < c.batch; k0 += T) {
      const int k = k0 + (int)threadIdx.x;
      below += __syncthreads_count(k < c.batch && first_item<P>(r, k) <= item);
    }
    b = max(below - 1, 0);
    nth = item - first_item<P>(r, b);
  } else {
    b = (int)(item / items_each);
    nth = item - items_each * b;
  }
  const AppendPlace p = place_of<P>(c, r, each, b, nth, head == 0 && !is_v && threadIdx.x == 0,
                                    new_lens, status);
  if (p.page < 0) return;
  const int64_t lo = p.lo, t0 = p.t0, end = p.end;
  const int len = p.len, page = p.page;

  const char *src = static_cast<const char *>(is_v ? r.v : r.k);
  const int64_t row_stride = is_v ? r.v_row_stride : r.k_row_stride;
  const int64_t head_stride = is_v ? r.v_head_stride : r.k_head_stride;
  constexpr int ES = DT == IBP_FP32 ? 4 : 2;
  float *scale_at = (is_v ? c.v_scales : c.k_scales) + (int64_t)page * c.n_heads + head;
  uint4 *codes = reinterpret_cast<uint4 *>(static_cast<char *>(is_v ? c.v_codes : c.k_codes) +
                                           kv_tile(c, page, head));
  const float before = t0 < len ? *scale_at : 0.0f;

  // tokens of the tile: [old, fresh) are the new rows
  const int old = (int)max((int64_t)len - t0, (int64_t)0), fresh = (int)min(end - t0, (int64_t)P);
  const int tok = threadIdx.x / GD;
  constexpr int STEP = Tile<P, D>::step;
  src += ((lo + (t0 - len) + tok) * row_stride + head * head_stride + (threadIdx.x % GD) * 16) * ES;
  codes += threadIdx.x;
  Raw16<DT> x[G];
  uint32_t bits = 0;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    x[g].clear();
    if (tok + g * STEP >= old && tok + g * STEP < fresh) x[g].load(src + g * (STEP * ES * row_stride));
  }
#pragma unroll
  for (int g = 0; g < G; ++g) bits = x[g].largest(bits);
  bits = block_max(Raw16<DT>::fold(bits), sm);
  float largest = Raw16<DT>::value(bits);
  const bool odd = bits >= Raw16<DT>::inf;  // infinities or NaN among the values
  if (odd) {
    float most = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) most = largest_finite<DT>(x[g], most);
    __syncthreads();
    largest = __uint_as_float(block_max(__float_as_uint(most), sm));
  }
  const float scale = fmaxf(before, kv_scale<CODE>(largest));
  const float inverse = kv_inverse(scale);
  if (threadIdx.x == 0) *scale_at = scale;
  if (!odd && scale < 0x1p120f) {
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (tok + g * STEP >= old && tok + g * STEP < fresh)
        codes[g * T] = encode16<DT, CODE, false>(x[g], inverse);
  } else {
#pragma unroll
    for (int g = 0; g < G; ++g)
      if (tok + g * STEP >= old && tok + g * STEP < fresh)
        codes[g * T] = encode16<DT, CODE, true>(x[g], inverse);
  }
  if (old && scale > before) {
    const float ratio = __fdiv_rn(before, scale);
    for (int g = 0; tok + g * STEP < old; ++g) codes[g * T] = rescale16<CODE>(codes[g * T], ratio);
  }
}

// The same for a few rows a sequence: one warp to a tile, which reads its rows twice
// (the second time from L1) and touches the codes that are there only when the scale
// grows. Bound by the chain of loads (offsets, length, table, scale and rows) and the
// launch: one token for each of 64 sequences, 8 heads of 128, takes 6.6 us.
constexpr int FEW_WARPS = 4;

template <int P, int D, int DT, int CODE>
__global__ void __launch_bounds__(32 * FEW_WARPS)
    kv_append_few_kernel(ibp_kv_cache c, ibp_kv_rows r, int64_t each, int64_t items_each,
                         int64_t items, int32_t *new_lens, int32_t *status) {
  constexpr int GD = D / 16;
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * FEW_WARPS + (threadIdx.x >> 5);
  const int64_t item = warp / (2 * c.n_heads);
  const int which = (int)(warp % (2 * c.n_heads)), head = which >> 1;
  const bool is_v = which & 1;
  if (item >= items) return;
  int b;
  int64_t nth;
  if (r.d_cu) {
    int below = 0;
    for (int k0 = 0; k0 < c.batch; k0 += 32)
      below += __popc(__ballot_sync(FULL, k0 + lane < c.batch && first_item<P>(r, k0 + lane) <= item));
    b = max(below - 1, 0);
    nth = item - first_item<P>(r, b);
  } else {
    b = (int)(item / items_each);
    nth = item - items_each * b;
  }
  const AppendPlace p = place_of<P>(c, r, each, b, nth, which == 0 && lane == 0, new_lens, status);
  if (p.page < 0) return;
  const char *src = static_cast<const char *>(is_v ? r.v : r.k);
  const int64_t row_stride = is_v ? r.v_row_stride : r.k_row_stride;
  const int64_t head_stride = is_v ? r.v_head_stride : r.k_head_stride;
  constexpr int ES = DT == IBP_FP32 ? 4 : 2;
  float *scale_at = (is_v ? c.v_scales : c.k_scales) + (int64_t)p.page * c.n_heads + head;
  uint4 *codes = reinterpret_cast<uint4 *>(static_cast<char *>(is_v ? c.v_codes : c.k_codes) +
                                           kv_tile(c, p.page, head));
  const float before = p.t0 < p.len ? *scale_at : 0.0f;
  const int64_t from = max(p.t0, (int64_t)p.len), to = min(p.end, p.t0 + P);
  const int groups = (int)(to - from) * GD, at0 = (int)(from - p.t0) * GD;
  src += ((p.lo + (from - p.len)) * row_stride + head * head_stride) * ES;
  auto load = [&](int i) {
    Raw16<DT> x;
    x.load(src + ((int64_t)(i / GD) * row_stride + (i % GD) * 16) * ES);
    return x;
  };
  uint32_t bits = 0;
  for (int i = lane; i < groups; i += 32) bits = load(i).largest(bits);
  bits = __reduce_max_sync(FULL, Raw16<DT>::fold(bits));
  float largest = Raw16<DT>::value(bits);
  const bool odd = bits >= Raw16<DT>::inf;
  if (odd) {
    float most = 0.0f;
    for (int i = lane; i < groups; i += 32) most = largest_finite<DT>(load(i), most);
    largest = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(most)));
  }
  const float scale = fmaxf(before, kv_scale<CODE>(largest));
  const float inverse = kv_inverse(scale);
  if (lane == 0) *scale_at = scale;
  if (!odd && scale < 0x1p120f)
    for (int i = lane; i < groups; i += 32) codes[at0 + i] = encode16<DT, CODE, false>(load(i), inverse);
  else
    for (int i = lane; i < groups; i += 32) codes[at0 + i] = encode16<DT, CODE, true>(load(i), inverse);
  if (scale > before) {
    const float ratio = __fdiv_rn(before, scale);
    for (int i = lane; i < at0; i += 32) codes[i] = rescale16<CODE>(codes[i], ratio);
  }
}

// value = rn(code * scale): bound by HBM (3 bytes an element in bf16). One CTA turns
// READ_TOKENS tokens of one head back into values; a thread moves 16 elements at a time,
// and the tokens need no exchange, so the split follows the output alone. 8 sequences of
// 4,096 tokens, 32 heads of 128 (805 MB moved): 122 us, 6.6 TB/s. (All loads of a thread
// ahead of its stores measured slower.)
constexpr int READ_TOKENS = 64;
constexpr int READ_THREADS = 128;

template <int D, int DT, int CODE>
__global__ void __launch_bounds__(READ_THREADS)
    kv_read_kernel(ibp_kv_cache c, int page_shift, const int32_t *begin, int64_t n_out,
                   void *k_out, void *v_out, int32_t *status) {
  constexpr int GD = D / 16, STEP = READ_THREADS / GD, ES = DT == IBP_FP32 ? 4 : 2;
  const int head = blockIdx.y % c.n_heads;
  const bool is_v = k_out == nullptr || (int)blockIdx.y >= c.n_heads;
  const int sub = threadIdx.x / GD, d0 = (threadIdx.x % GD) * 16, b = blockIdx.z;
  const char *codes = static_cast<const char *>(is_v ? c.v_codes : c.k_codes);
  const float *scales = is_v ? c.v_scales : c.k_scales;
  const int len = kv_len(c, b, status);
  const int64_t i0 = (int64_t)blockIdx.x * READ_TOKENS + sub;
  // without a sign: a token before the sequence wraps to one far past it, and none wraps back
  // (the sums are above -2^31 and below 2^31 + 2^30)
  const uint32_t first = (begin ? (uint32_t)__ldg(begin + b) : 0u) + (uint32_t)i0;
  char *out = static_cast<char *>(is_v ? v_out : k_out) +
              ((((int64_t)b * n_out + i0) * c.n_heads + head) * D + d0) * ES;
  const int left = (int)min(n_out - i0, (int64_t)READ_TOKENS);
  const int64_t out_step = (int64_t)STEP * c.n_heads * D * ES;
#pragma unroll
  for (int k = 0; k < READ_TOKENS; k += STEP, out += out_step) {
    if (k >= left) break;
    const uint32_t t = first + k;
    float x[16] = {};
    if (t < (uint32_t)len) {
      const int page = kv_page(c, b, (int)(t >> page_shift), status);
      if (page >= 0) {
        const int64_t tile = (int64_t)page * c.n_heads + head;
        const float scale = __ldg(scales + tile);
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(
            codes + ((tile << page_shift) + (t & (c.page_tokens - 1))) * D + d0));
        kv_decode4<CODE>(w.x, x);
        kv_decode4<CODE>(w.y, x + 4);
        kv_decode4<CODE>(w.z, x + 8);
        kv_decode4<CODE>(w.w, x + 12);
#pragma unroll
        for (int e = 0; e < 16; e += 4) mul4(x + e, scale);
      }
    }
    store16<DT>(out, x);
  }
}

template <int P, int D, int DT>
int append_code(const ibp_kv_cache &c, const ibp_kv_rows &r, int32_t *new_lens, int32_t *status,
                cudaStream_t s) {
  const int64_t each = r.d_cu ? 0 : r.n_rows / c.batch;
  const int64_t items_each = each > 0 ? (each - 1) / P + 2 : 1;
  const int64_t items = r.d_cu ? r.n_rows / P + 2 * (int64_t)c.batch : items_each * c.batch;
  if (items > 0x7FFFFFFF) return IBP_ERR_UNSUPPORTED;
  // A warp to a tile while a sequence brings less than a quarter of a page: no barrier, and
  // a quarter as many CTAs, but a warp takes more rows in turn. One token for each of 64
  // sequences, 8 heads of 128: 6.6 us, with a CTA to a tile 9.3 (alone, cold). In pages of 64,
  // calls of 64 sequences: 8 rows each 8.9 us | 10.9 with a CTA, 24 rows 10.9 | 10.9; of 8
  // sequences: 15 rows 8.9 | 8.9, 24 rows 10.9 | 8.9, 64 rows 13.0 | 8.9.
  if (r.n_rows < (int64_t)c.batch * (P / 4)) {
    const int64_t ctas = (items * 2 * c.n_heads + FEW_WARPS - 1) / FEW_WARPS;
    if (ctas > 0x7FFFFFFF) return IBP_ERR_UNSUPPORTED;
    const auto kernel = c.code == IBP_KV_INT8 ? kv_append_few_kernel<P, D, DT, IBP_KV_INT8>
                                              : kv_append_few_kernel<P, D, DT, IBP_KV_E4M3>;
    kernel<<<(unsigned)ctas, 32 * FEW_WARPS, 0, s>>>(c, r, each, items_each, items, new_lens, status);
  } else {
    const dim3 grid((unsigned)items, (unsigned)c.n_heads, 2);
    const auto kernel = c.code == IBP_KV_INT8 ? kv_append_kernel<P, D, DT, IBP_KV_INT8>
                                              : kv_append_kernel<P, D, DT, IBP_KV_E4M3>;
    kernel<<<grid, Tile<P, D>::threads, 0, s>>>(c, r, each, items_each, new_lens, status);
  }
  return cudaGetLastError() == cudaSuccess ? IBP_OK : IBP_ERR_CUDA;
}

template <int P, int D>
int append_dtype(const ibp_kv_cache &c, const ibp_kv_rows &r, int32_t *new_lens, int32_t *status,
                 cudaStream_t s) {
  switch (r.dtype) {
    case IBP_FP32: return append_code<P, D, IBP_FP32>(c, r, new_lens, status, s);
    case IBP_FP16: return append_code<P, D, IBP_FP16>(c, r, new_lens, status, s);
    default: return append_code<P, D, IBP_BF16>(c, r, new_lens, status, s);
  }
}

template <int P>
int append_dim(const ibp_kv_cache &c, const ibp_kv_rows &r, int32_t *new_lens, int32_t *status,
               cudaStream_t s) {
  return c.head_dim == 64 ? append_dtype<P, 64>(c, r, new_lens, status, s)
                          : append_dtype<P, 128>(c, r, new_lens, status, s);
}

template <int D, int DT>
int read_code(const ibp_kv_cache &c, const int32_t *begin, int64_t n_out, void *k_out, void *v_out,
              int32_t *status, cudaStream_t s) {
  const int64_t chunks = (n_out + READ_TOKENS - 1) / READ_TOKENS;
  if (chunks > 0x7FFFFFFF) return IBP_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)chunks, (unsigned)(c.n_heads * ((k_out != nullptr) + (v_out != nullptr))),
                  (unsigned)c.batch);
  const int shift = c.page_tokens == 16 ? 4 : c.page_tokens == 32 ? 5 : c.page_tokens == 64 ? 6 : 7;
  const auto kernel = c.code == IBP_KV_INT8 ? kv_read_kernel<D, DT, IBP_KV_INT8>
                                            : kv_read_kernel<D, DT, IBP_KV_E4M3>;
  kernel<<<grid, READ_THREADS, 0, s>>>(c, shift, begin, n_out, k_out, v_out, status);
  return cudaGetLastError() == cudaSuccess ? IBP_OK : IBP_ERR_CUDA;
}

template <int D>
int read_dtype(const ibp_kv_cache &c, const int32_t *begin, int64_t n_out, void *k_out, void *v_out,
               int dtype, int32_t *status, cudaStream_t s) {
  switch (dtype) {
    case IBP_FP32: return read_code<D, IBP_FP32>(c, begin, n_out, k_out, v_out, status, s);
    case IBP_FP16: return read_code<D, IBP_FP16>(c, begin, n_out, k_out, v_out, status, s);
    default: return read_code<D, IBP_BF16>(c, begin, n_out, k_out, v_out, status, s);
  }
}

}  // namespace

int launch_kv_append(const ibp_kv_cache &c, const ibp_kv_rows &r, int32_t *d_new_lens,
                     int32_t *d_status, cudaStream_t s) {
  switch (c.page_tokens) {
    case 16: return append_dim<16>(c, r, d_new_lens, d_status, s);
    case 32: return append_dim<32>(c, r, d_new_lens, d_status, s);
    case 64: return append_dim<64>(c, r, d_new_lens, d_status, s);
    default: return append_dim<128>(c, r, d_new_lens, d_status, s);
  }
}

int launch_kv_read(const ibp_kv_cache &c, const int32_t *d_begin, int64_t n_out, void *k_out,
                   void *v_out, int dtype, int32_t *d_status, cudaStream_t s) {
  return c.head_dim == 64 ? read_dtype<64>(c, d_begin, n_out, k_out, v_out, dtype, d_status, s)
                          : read_dtype<128>(c, d_begin, n_out, k_out, v_out, dtype, d_status, s);
}

}  // namespace ibp
