// Append and read of the 8-bit paged key/value cache (declared in include/ibp.h).
#include "ibp_kv_device.cuh"

namespace ibp {

namespace {

// One CTA quantises what one (page, head) tile of K or V receives. A thread holds G
// groups of 16 consecutive elements of a token, so its source comes in 16-byte loads
// and its codes leave in 16-byte stores; the tile's values stay in registers between
// the maximum and the rounding, so rows are read once and codes written once.
template <int P, int D>
struct Tile {
  static constexpr int groups = P * D / 16;
  static constexpr int threads = groups < 256 ? groups : 256;
  static constexpr int per_thread = groups / threads;
};

// Work item -> (sequence, page): sequence b's items start at cu[b]/P + 2b (its rows
// touch at most (rows - 1)/P + 2 pages, so items of two sequences never overlap).
template <int P, int D, int DT, int CODE>
__global__ void __launch_bounds__(Tile<P, D>::threads)
    kv_append_kernel(ibp_kv_cache c, ibp_kv_rows r, int64_t each, int64_t items_each,
                     int32_t *new_lens, int32_t *status) {
  constexpr int T = Tile<P, D>::threads, G = Tile<P, D>::per_thread, GD = D / 16;
  __shared__ float sm[32];
  const int64_t item = blockIdx.x;
  const int head = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  int b;
  int64_t first_item;
  if (r.d_cu) {
    // starts rise with b: the last one that is not past the item
    int below = 0;
    for (int k0 = 0; k0 < c.batch; k0 += T) {
      const int k = k0 + (int)threadIdx.x;
      below += __syncthreads_count(k < c.batch &&
                                   max(__ldg(r.d_cu + k), 0) / P + 2 * (int64_t)k <= item);
    }
    b = max(below - 1, 0);
    first_item = max(__ldg(r.d_cu + b), 0) / P + 2 * (int64_t)b;
  } else {
    b = (int)(item / items_each);
    first_item = items_each * b;
  }
  int64_t lo, hi;
  kv_row_range(r.d_cu, r.n_rows, each, b, status, &lo, &hi);
  const int len = kv_len(c, b, status);
  const int64_t cap = (int64_t)c.table_cols * P;
  const int64_t all = len + (hi - lo), end = all < cap ? all : cap;
  const int64_t nth = item - first_item;
  if (nth < 0) return;
  if (nth == 0 && head == 0 && !is_v && threadIdx.x == 0) {
    if (end != all) report(status, IBP_ERR_INDEX);
    if (new_lens) new_lens[b] = (int32_t)end;
  }
  const int64_t t0 = (len / P + nth) * P;
  if (t0 >= end || hi == lo) return;
  const int page = kv_page(c, b, (int)(t0 / P), status);
  if (page < 0) return;

  const char *src = static_cast<const char *>(is_v ? r.v : r.k);
  const int64_t row_stride = is_v ? r.v_row_stride : r.k_row_stride;
  const int64_t head_stride = is_v ? r.v_head_stride : r.k_head_stride;
  constexpr int ES = DT == IBP_FP32 ? 4 : 2;
  float *scale_at = (is_v ? c.v_scales : c.k_scales) + (int64_t)page * c.n_heads + head;
  uint4 *codes = reinterpret_cast<uint4 *>(static_cast<char *>(is_v ? c.v_codes : c.k_codes) +
                                           kv_tile(c, page, head));
  const float before = t0 < len ? *scale_at : 0.0f;

  float x[G][16];
  float largest = 0.0f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int at = g * T + (int)threadIdx.x;
    const int64_t t = t0 + at / GD;
    if (t >= len && t < end) {
      load16<DT>(src + ((lo + (t - len)) * row_stride + head * head_stride + (at % GD) * 16) * ES, x[g]);
#pragma unroll
      for (int i = 0; i < 16; ++i) largest = fmaxf(largest, finite_abs(x[g][i]));
    }
  }
  largest = block_max(largest, sm);
  const float scale = fmaxf(before, kv_scale<CODE>(largest));
  const float inverse = kv_inverse(scale);
  const bool grew = scale > before;
  const float ratio = grew ? __fdiv_rn(before, scale) : 1.0f;
  if (threadIdx.x == 0) *scale_at = scale;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int at = g * T + (int)threadIdx.x;
    const int64_t t = t0 + at / GD;
    if (t >= end || (t < len && !grew)) continue;
    uint32_t w[4];
    if (t >= len) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = kv_encode4<CODE>(__fmul_rn(x[g][4 * i], inverse), __fmul_rn(x[g][4 * i + 1], inverse),
                                __fmul_rn(x[g][4 * i + 2], inverse),
                                __fmul_rn(x[g][4 * i + 3], inverse));
    } else {
      const uint4 old = codes[at];
      const uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float y[4];
        kv_decode4<CODE>(o[i], y);
        w[i] = kv_encode4<CODE>(__fmul_rn(y[0], ratio), __fmul_rn(y[1], ratio),
                                __fmul_rn(y[2], ratio), __fmul_rn(y[3], ratio));
      }
    }
    codes[at] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// One CTA turns READ_TOKENS tokens of one head back into values; a thread moves 16
// elements at a time.
constexpr int READ_TOKENS = 64;
constexpr int READ_THREADS = 128;

template <int D, int DT, int CODE>
__global__ void __launch_bounds__(READ_THREADS)
    kv_read_kernel(ibp_kv_cache c, const int32_t *begin, int64_t n_out, void *k_out, void *v_out,
                   int32_t *status) {
  constexpr int GD = D / 16, STEP = READ_THREADS / GD, ES = DT == IBP_FP32 ? 4 : 2;
  const int head = blockIdx.y % c.n_heads;
  const bool is_v = k_out == nullptr || (int)blockIdx.y >= c.n_heads;
  const int sub = threadIdx.x / GD, d0 = (threadIdx.x % GD) * 16;
  const char *codes = static_cast<const char *>(is_v ? c.v_codes : c.k_codes);
  const float *scales = is_v ? c.v_scales : c.k_scales;
  char *out = static_cast<char *>(is_v ? v_out : k_out);
  const int b = blockIdx.z;
  const int len = kv_len(c, b, status);
  const int64_t from = begin ? __ldg(begin + b) : 0;
#pragma unroll
  for (int k = 0; k < READ_TOKENS; k += STEP) {
    const int64_t i = (int64_t)blockIdx.x * READ_TOKENS + k + sub;
    if (i >= n_out) break;
    const int64_t t = from + i;
    float x[16] = {};
    if (t >= 0 && t < len) {
      const int page = kv_page(c, b, (int)(t / c.page_tokens), status);
      if (page >= 0) {
        const float scale = __ldg(scales + (int64_t)page * c.n_heads + head);
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(
            codes + kv_tile(c, page, head) + (t % c.page_tokens) * D + d0));
        kv_decode4<CODE>(w.x, x);
        kv_decode4<CODE>(w.y, x + 4);
        kv_decode4<CODE>(w.z, x + 8);
        kv_decode4<CODE>(w.w, x + 12);
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = __fmul_rn(x[e], scale);
      }
    }
    store16<DT>(out + ((((int64_t)b * n_out + i) * c.n_heads + head) * D + d0) * ES, x);
  }
}

template <int P, int D, int DT>
int append_code(const ibp_kv_cache &c, const ibp_kv_rows &r, int32_t *new_lens, int32_t *status,
                cudaStream_t s) {
  const int64_t each = r.d_cu ? 0 : r.n_rows / c.batch;
  const int64_t items_each = each > 0 ? (each - 1) / P + 2 : 1;
  const int64_t items = r.d_cu ? r.n_rows / P + 2 * (int64_t)c.batch : items_each * c.batch;
  if (items > 0x7FFFFFFF) return IBP_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)items, (unsigned)c.n_heads, 2);
  if (c.code == IBP_KV_INT8)
    kv_append_kernel<P, D, DT, IBP_KV_INT8>
        <<<grid, Tile<P, D>::threads, 0, s>>>(c, r, each, items_each, new_lens, status);
  else
    kv_append_kernel<P, D, DT, IBP_KV_E4M3>
        <<<grid, Tile<P, D>::threads, 0, s>>>(c, r, each, items_each, new_lens, status);
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
  if (c.code == IBP_KV_INT8)
    kv_read_kernel<D, DT, IBP_KV_INT8><<<grid, READ_THREADS, 0, s>>>(c, begin, n_out, k_out, v_out, status);
  else
    kv_read_kernel<D, DT, IBP_KV_E4M3><<<grid, READ_THREADS, 0, s>>>(c, begin, n_out, k_out, v_out, status);
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
