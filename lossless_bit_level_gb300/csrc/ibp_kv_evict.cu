// Eviction from the 8-bit paged key/value cache by accumulated attention weight
// (declared in include/ibp.h): which tokens stay, then their values requantised into
// the destination's pages.
#include "ibp_kv_device.cuh"

namespace ibp {

namespace {

constexpr int SELECT_THREADS = 1024;

// Unsigned order of the weights: a larger key is a larger weight, NaN lowest, -0 = 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.0f ? 0.0f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the block; *total gets the sum. `sm`: 33 words.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *sm, uint32_t *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(FULL, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t y = lane < (int)(blockDim.x >> 5) ? sm[lane] : 0u, z = y;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(FULL, z, o);
      if (lane >= o) z += u;
    }
    sm[lane] = z - y;
    if (lane == 31) sm[32] = z;
  }
  __syncthreads();
  const uint32_t r = sm[warp] + x - v;
  *total = sm[32];
  __syncthreads();
  return r;
}

// One CTA per (sequence, head): the k-th largest key by four passes of 8-bit counts,
// then one pass in token order that lists the tokens above it and the first of those
// equal to it.
__global__ void __launch_bounds__(SELECT_THREADS)
    kv_select_kernel(ibp_kv_cache c, const float *weights, int64_t stride, int budget, int recent,
                     int32_t *new_lens, float *new_weights, int64_t new_stride, int32_t *kept_out,
                     int32_t *list, int32_t *status) {
  __shared__ uint32_t hist[256], sm[33], chosen[2];
  const int head = blockIdx.x % c.n_heads, b = blockIdx.x / c.n_heads;
  const int64_t bh = (int64_t)b * c.n_heads + head;
  const float *w = weights + bh * stride;
  const int len = kv_len(c, b, status), out = min(len, budget);
  const bool all = len <= budget;
  const int open = all ? 0 : len - recent;  // tokens that compete
  uint32_t need = all ? 0u : (uint32_t)(budget - recent), prefix = 0;
  if (need) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += SELECT_THREADS) hist[i] = 0;
      __syncthreads();
      const uint32_t above = shift == 24 ? 0u : FULL << (shift + 8);
      for (int t = threadIdx.x; t < open; t += SELECT_THREADS) {
        const uint32_t key = weight_key(w[t]);
        if (((key ^ prefix) & above) == 0) atomicAdd(&hist[(key >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        uint32_t left = need;
        int d = 255;
        while (d > 0 && hist[d] < left) left -= hist[d--];
        chosen[0] = (uint32_t)d;
        chosen[1] = left;
      }
      __syncthreads();
      prefix |= chosen[0] << shift;
      need = chosen[1];
    }
  }
  // need: how many of the tokens whose key equals `prefix` stay
  const bool any = !all && budget > recent;
  uint32_t base = 0, equal_base = 0;
  int32_t *row = list + bh * budget;
  for (int t0 = 0; t0 < len; t0 += SELECT_THREADS) {
    const int t = t0 + (int)threadIdx.x;
    bool keep = t < len, equal = false;
    if (keep && !all && t < open) {
      const uint32_t key = weight_key(w[t]);
      equal = any && key == prefix;
      keep = any && key > prefix;
    }
    uint32_t equals, kept;
    const uint32_t before = block_scan(equal, sm, &equals);
    if (equal) keep = equal_base + before < need;
    equal_base += equals;
    const uint32_t at = base + block_scan(keep, sm, &kept);
    base += kept;
    if (keep && at < (uint32_t)out) {
      row[at] = t;
      if (kept_out) kept_out[bh * budget + at] = t;
      if (new_weights) new_weights[bh * new_stride + at] = w[t];
    }
  }
  for (int64_t i = out + (int)threadIdx.x; i < budget; i += SELECT_THREADS)
    if (kept_out) kept_out[bh * budget + i] = -1;
  if (new_weights)
    for (int64_t i = out + (int)threadIdx.x; i < new_stride; i += SELECT_THREADS)
      new_weights[bh * new_stride + i] = 0.0f;
  if (head == 0 && threadIdx.x == 0) new_lens[b] = out;
}

// One CTA per (sequence, head, destination page, K or V): the kept tokens' values,
// their maximum, their codes.
template <int P, int D, int CODE>
__global__ void __launch_bounds__(P *D / 16 < 256 ? P * D / 16 : 256)
    kv_move_kernel(ibp_kv_cache c, ibp_kv_cache dst, int budget, const int32_t *list,
                   int32_t *status) {
  constexpr int T = P * D / 16 < 256 ? P * D / 16 : 256, G = P * D / 16 / T, GD = D / 16;
  __shared__ float sm[32];
  const int head = blockIdx.y % c.n_heads;
  const bool is_v = (int)blockIdx.y >= c.n_heads;
  const int t0 = blockIdx.x * P;
  const int b = blockIdx.z;
  const int out = min(kv_len(c, b, nullptr), budget);
  if (t0 >= out) return;
  const int to = kv_page(dst, b, blockIdx.x, status);
  if (to < 0) return;
  const int32_t *row = list + ((int64_t)b * c.n_heads + head) * budget;
  const char *codes = static_cast<const char *>(is_v ? c.v_codes : c.k_codes);
  const float *scales = is_v ? c.v_scales : c.k_scales;
  float x[G][16], largest = 0.0f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int at = g * T + (int)threadIdx.x, t = t0 + at / GD;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[g][i] = 0.0f;
    if (t < out) {
      const int from = __ldg(row + t);
      const int page = kv_page(c, b, from / P, status);
      if (page >= 0) {
        const float scale = __ldg(scales + (int64_t)page * c.n_heads + head);
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(
            codes + kv_tile(c, page, head) + (from % P) * D + (at % GD) * 16));
        kv_decode4<CODE>(w.x, x[g]);
        kv_decode4<CODE>(w.y, x[g] + 4);
        kv_decode4<CODE>(w.z, x[g] + 8);
        kv_decode4<CODE>(w.w, x[g] + 12);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          x[g][i] = __fmul_rn(x[g][i], scale);
          largest = fmaxf(largest, finite_abs(x[g][i]));
        }
      }
    }
  }
  largest = block_max(largest, sm);
  const float scale = kv_scale<CODE>(largest), inverse = kv_inverse(scale);
  if (threadIdx.x == 0)
    (is_v ? dst.v_scales : dst.k_scales)[(int64_t)to * c.n_heads + head] = scale;
  uint4 *put = reinterpret_cast<uint4 *>(static_cast<char *>(is_v ? dst.v_codes : dst.k_codes) +
                                         kv_tile(dst, to, head));
#pragma unroll
  for (int g = 0; g < G; ++g) {
    const int at = g * T + (int)threadIdx.x, t = t0 + at / GD;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = kv_encode4<CODE>(__fmul_rn(x[g][4 * i], inverse), __fmul_rn(x[g][4 * i + 1], inverse),
                              __fmul_rn(x[g][4 * i + 2], inverse),
                              __fmul_rn(x[g][4 * i + 3], inverse));
    if (t < out) put[at] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int P, int D>
int move_code(const ibp_kv_cache &c, const ibp_kv_cache &dst, int budget, const int32_t *list,
              int32_t *status, cudaStream_t s) {
  const int64_t cap = (int64_t)c.table_cols * P;
  const dim3 grid((unsigned)(((budget < cap ? budget : cap) + P - 1) / P), (unsigned)(2 * c.n_heads),
                  (unsigned)c.batch);
  constexpr int T = P * D / 16 < 256 ? P * D / 16 : 256;
  if (c.code == IBP_KV_INT8)
    kv_move_kernel<P, D, IBP_KV_INT8><<<grid, T, 0, s>>>(c, dst, budget, list, status);
  else
    kv_move_kernel<P, D, IBP_KV_E4M3><<<grid, T, 0, s>>>(c, dst, budget, list, status);
  return cudaGetLastError() == cudaSuccess ? IBP_OK : IBP_ERR_CUDA;
}

template <int P>
int move_dim(const ibp_kv_cache &c, const ibp_kv_cache &dst, int budget, const int32_t *list,
             int32_t *status, cudaStream_t s) {
  return c.head_dim == 64 ? move_code<P, 64>(c, dst, budget, list, status, s)
                          : move_code<P, 128>(c, dst, budget, list, status, s);
}

}  // namespace

size_t kv_evict_scratch_bytes(const ibp_kv_cache &c, int64_t budget) {
  return ((size_t)c.batch * c.n_heads * budget * sizeof(int32_t) + 15) / 16 * 16;
}

int launch_kv_evict(const ibp_kv_cache &c, const float *d_weights, int64_t weights_stride,
                    int64_t budget, int64_t recent, const ibp_kv_cache &dst, int32_t *d_new_lens,
                    float *d_new_weights, int64_t new_weights_stride, int32_t *d_kept,
                    void *d_scratch, int32_t *d_status, cudaStream_t s) {
  int32_t *list = static_cast<int32_t *>(d_scratch);
  kv_select_kernel<<<(unsigned)(c.batch * c.n_heads), SELECT_THREADS, 0, s>>>(
      c, d_weights, weights_stride, (int)budget, (int)recent, d_new_lens, d_new_weights,
      new_weights_stride, d_kept, list, d_status);
  if (cudaGetLastError() != cudaSuccess) return IBP_ERR_CUDA;
  switch (c.page_tokens) {
    case 16: return move_dim<16>(c, dst, (int)budget, list, d_status, s);
    case 32: return move_dim<32>(c, dst, (int)budget, list, d_status, s);
    case 64: return move_dim<64>(c, dst, (int)budget, list, d_status, s);
    default: return move_dim<128>(c, dst, (int)budget, list, d_status, s);
  }
}

}  // namespace ibp
