// Attention over the 8-bit paged key/value cache (declared in include/ibp.h).
//
// out = sum_t p_t v_t, p = softmax of scale * q . k_t over the tokens a row sees. One
// pass over the keys with the running maximum m and sum l of the softmax:
//   m' = max(m, x), l' = l 2^(m - m') + 2^(x - m'), o' = o 2^(m - m') + 2^(x - m') v
// with x in units of log2(e).
#include "ibp_kv_device.cuh"

namespace ibp {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr int WARPS = 4;

template <int DT, int N>
__device__ __forceinline__ void load_few(const char *p, float *x) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint32_t u = *reinterpret_cast<const uint32_t *>(p + 2 * i);
    if constexpr (DT == IBP_BF16) {
      x[i] = __uint_as_float(u << 16);
      x[i + 1] = __uint_as_float(u & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
      x[i] = f.x;
      x[i + 1] = f.y;
    }
  }
}

template <int CODE, int N>
__device__ __forceinline__ void load_codes(const char *p, float *x) {
  const uint32_t w = N == 4 ? *reinterpret_cast<const uint32_t *>(p)
                            : *reinterpret_cast<const uint16_t *>(p);
  float y[4];
  kv_decode4<CODE>(w, y);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = y[i];
}

// One CTA per (query row, query head, sequence); its warps take every fourth key.
template <int D, int DT, int CODE>
__global__ void __launch_bounds__(32 * WARPS)
    kv_attention_kernel(ibp_kv_cache c, ibp_kv_query q, float *lse2, int32_t *status) {
  constexpr int N = D / 32;
  __shared__ float sm_o[WARPS][D], sm_m[WARPS], sm_l[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qh = blockIdx.y, group = q.q_heads / c.n_heads, head = qh / group;
  const char *kc = static_cast<const char *>(c.k_codes), *vc = static_cast<const char *>(c.v_codes);
  for (int b = blockIdx.z; b < c.batch; b += gridDim.z) {
    int64_t lo, hi;
    kv_row_range(q.d_cu, q.n_rows, q.max_q, b, status, &lo, &hi);
    const int64_t n = hi - lo, i = blockIdx.x;
    if (n > q.max_q) report(status, IBP_ERR_INDEX);
    if (i >= n) continue;
    const int len = kv_len(c, b, status);
    const int limit = (int)max((int64_t)0, len - n + i + 1);
    float qv[N], o[N] = {}, m = -INFINITY, l = 0.0f;
    load_few<DT, N>(static_cast<const char *>(q.q) +
                        2 * ((lo + i) * q.q_row_stride + qh * q.q_head_stride + lane * N),
                    qv);
    for (int t = warp; t < limit; t += WARPS) {
      const int page = kv_page(c, b, t / c.page_tokens, status);
      if (page < 0) continue;
      const int64_t at = kv_tile(c, page, head) + (t % c.page_tokens) * D + lane * N;
      const int64_t st = (int64_t)page * c.n_heads + head;
      float k[N], v[N], x = 0.0f;
      load_codes<CODE, N>(kc + at, k);
      load_codes<CODE, N>(vc + at, v);
#pragma unroll
      for (int e = 0; e < N; ++e) x = fmaf(qv[e], k[e], x);
      for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(FULL, x, w);
      x *= __ldg(c.k_scales + st) * (q.scale * LOG2E);
      const float to = fmaxf(m, x), keep = exp2f(m - to), p = exp2f(x - to);
      const float pv = p * __ldg(c.v_scales + st);
      m = to;
      l = l * keep + p;
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = o[e] * keep + pv * v[e];
    }
    if (lane == 0) {
      sm_m[warp] = m;
      sm_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) sm_o[warp][lane * N + e] = o[e];
    __syncthreads();
    float top = -INFINITY, sum = 0.0f;
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, sm_m[w]);
    if (top == -INFINITY) top = 0.0f;
    for (int w = 0; w < WARPS; ++w) sum += sm_l[w] * exp2f(sm_m[w] - top);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const int64_t row = (lo + i) * q.q_heads + qh;
    if (threadIdx.x < D / 2) {
      float y[2] = {};
      for (int w = 0; w < WARPS; ++w)
        for (int e = 0; e < 2; ++e)
          y[e] += sm_o[w][2 * threadIdx.x + e] * exp2f(sm_m[w] - top);
      uint32_t *out = reinterpret_cast<uint32_t *>(
          static_cast<char *>(q.out) + 2 * ((lo + i) * q.out_row_stride + qh * q.out_head_stride));
      out[threadIdx.x] = pack2<DT>(y[0] * inv, y[1] * inv);
    }
    if (threadIdx.x == 0) {
      const float z = sum > 0.0f ? top + log2f(sum) : -INFINITY;
      lse2[row] = z;
      if (q.d_lse) q.d_lse[row] = z * LN2;
    }
    __syncthreads();
  }
}

// weights[t] = decay * weights_in[t] + the sum over rows and heads of 2^(x - lse2).
template <int D, int DT, int CODE>
__global__ void __launch_bounds__(128)
    kv_weights_kernel(ibp_kv_cache c, ibp_kv_query q, const float *lse2, int32_t *status) {
  const int head = blockIdx.y, group = q.q_heads / c.n_heads;
  for (int b = blockIdx.z; b < c.batch; b += gridDim.z) {
    int64_t lo, hi;
    kv_row_range(q.d_cu, q.n_rows, q.max_q, b, status, &lo, &hi);
    const int len = kv_len(c, b, status), t = blockIdx.x * 128 + threadIdx.x;
    if (t >= len) continue;
    const int page = kv_page(c, b, t / c.page_tokens, status);
    float k[D], sum = 0.0f;
    if (page >= 0) {
      const uint4 *p = reinterpret_cast<const uint4 *>(
          static_cast<const char *>(c.k_codes) + kv_tile(c, page, head) + (t % c.page_tokens) * D);
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        const uint4 w = p[e];
        kv_decode4<CODE>(w.x, k + 16 * e);
        kv_decode4<CODE>(w.y, k + 16 * e + 4);
        kv_decode4<CODE>(w.z, k + 16 * e + 8);
        kv_decode4<CODE>(w.w, k + 16 * e + 12);
      }
      const float f = __ldg(c.k_scales + (int64_t)page * c.n_heads + head) * (q.scale * LOG2E);
      for (int64_t i = 0; i < min(hi - lo, q.max_q); ++i) {
        if (t >= len - (hi - lo) + i + 1) continue;
        for (int g = 0; g < group; ++g) {
          const int qh = head * group + g;
          const char *row = static_cast<const char *>(q.q) +
                            2 * ((lo + i) * q.q_row_stride + qh * q.q_head_stride);
          float x = 0.0f;
#pragma unroll
          for (int e = 0; e < D; e += 4) {
            float y[4];
            load_few<DT, 4>(row + 2 * e, y);
#pragma unroll
            for (int w = 0; w < 4; ++w) x = fmaf(y[w], k[e + w], x);
          }
          sum += exp2f(x * f - lse2[(lo + i) * q.q_heads + qh]);
        }
      }
    }
    const int64_t at = ((int64_t)b * c.n_heads + head) * q.weights_stride + t;
    q.d_weights[at] = (q.d_weights_in ? q.decay * q.d_weights_in[at] : 0.0f) + sum;
  }
}

template <int D, int DT, int CODE>
int launch_for(const ibp_kv_cache &c, const ibp_kv_query &q, void *scratch, int32_t *status,
               cudaStream_t s) {
  float *lse2 = static_cast<float *>(scratch);
  const unsigned z = (unsigned)c.batch;
  kv_attention_kernel<D, DT, CODE>
      <<<dim3((unsigned)q.max_q, (unsigned)q.q_heads, z), 32 * WARPS, 0, s>>>(c, q, lse2, status);
  if (q.d_weights) {
    const unsigned tiles = (unsigned)((c.table_cols * c.page_tokens + 127) / 128);
    kv_weights_kernel<D, DT, CODE>
        <<<dim3(tiles, (unsigned)c.n_heads, z), 128, 0, s>>>(c, q, lse2, status);
  }
  return cudaGetLastError() == cudaSuccess ? IBP_OK : IBP_ERR_CUDA;
}

template <int D, int DT>
int launch_code(const ibp_kv_cache &c, const ibp_kv_query &q, void *scratch, int32_t *status,
                cudaStream_t s) {
  return c.code == IBP_KV_INT8 ? launch_for<D, DT, IBP_KV_INT8>(c, q, scratch, status, s)
                               : launch_for<D, DT, IBP_KV_E4M3>(c, q, scratch, status, s);
}

template <int D>
int launch_dtype(const ibp_kv_cache &c, const ibp_kv_query &q, void *scratch, int32_t *status,
                 cudaStream_t s) {
  return q.dtype == IBP_BF16 ? launch_code<D, IBP_BF16>(c, q, scratch, status, s)
                             : launch_code<D, IBP_FP16>(c, q, scratch, status, s);
}

}  // namespace

size_t kv_attention_scratch_bytes(const ibp_kv_cache &c, int64_t n_rows, int64_t max_q,
                                  int q_heads, bool with_weights) {
  return ((size_t)n_rows * q_heads * sizeof(float) + 15) / 16 * 16;
}

int launch_kv_attention(const ibp_kv_cache &c, const ibp_kv_query &q, void *d_scratch,
                        int32_t *d_status, cudaStream_t s) {
  return c.head_dim == 64 ? launch_dtype<64>(c, q, d_scratch, d_status, s)
                          : launch_dtype<128>(c, q, d_scratch, d_status, s);
}

}  // namespace ibp
