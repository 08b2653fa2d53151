// Device-side helpers of the 8-bit paged key/value cache kernels: lengths and page
// lookups with their checks, the quantisation rule, code <-> float.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <float.h>

#include "ibp_device.cuh"
#include "ibp_kv.h"

namespace ibp {

// Tokens sequence b holds, clamped to its capacity.
__device__ __forceinline__ int kv_len(const ibp_kv_cache &c, int b, int32_t *status) {
  const int n = __ldg(c.d_lens + b), cap = c.table_cols * c.page_tokens;
  const int m = min(max(n, 0), cap);
  if (m != n) report(status, IBP_ERR_INDEX);
  return m;
}

// Rows [lo, hi) of sequence b; cu null: `each` rows a sequence.
__device__ __forceinline__ void kv_row_range(const int32_t *cu, int64_t n_rows, int64_t each, int b,
                                             int32_t *status, int64_t *lo, int64_t *hi) {
  if (!cu) {
    *lo = each * b;
    *hi = *lo + each;
    return;
  }
  const int64_t x = __ldg(cu + b), y = __ldg(cu + b + 1);
  *lo = min(max(x, (int64_t)0), n_rows);
  *hi = min(max(y, *lo), n_rows);
  if (*lo != x || *hi != y) report(status, IBP_ERR_INDEX);
}

// Page `col` of sequence b, or -1 (recorded) for an id outside the pool.
__device__ __forceinline__ int kv_page(const ibp_kv_cache &c, int b, int col, int32_t *status) {
  const int p = __ldg(c.d_table + (int64_t)b * c.table_stride + col);
  if (p >= 0 && p < c.n_pages) return p;
  report(status, IBP_ERR_INDEX);
  return -1;
}

// First byte of the (page, head) tile.
__device__ __forceinline__ int64_t kv_tile(const ibp_kv_cache &c, int page, int head) {
  return ((int64_t)page * c.n_heads + head) * c.page_tokens * c.head_dim;
}

template <int CODE>
struct KvQmax {
  static constexpr float value = CODE == IBP_KV_INT8 ? 127.0f : 448.0f;
};

// Scale of a tile whose largest finite magnitude is `largest`, and its inverse.
template <int CODE>
__device__ __forceinline__ float kv_scale(float largest) {
  if (!(largest > 0.0f)) return 0.0f;
  return fminf(fmaxf(__fmul_rn(largest, 1.0f / KvQmax<CODE>::value), 0x1p-100f), 0x1p120f);
}
__device__ __forceinline__ float kv_inverse(float scale) {
  return scale > 0.0f ? __fdiv_rn(1.0f, scale) : 0.0f;
}

// |x|, or 0 where x is an infinity or NaN.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? a : 0.0f;
}

// Four values (already times the inverse scale) to four codes in one word. int8:
// adding 1.5 * 2^23 leaves the value rounded to nearest even in the low byte.
template <int CODE>
__device__ __forceinline__ uint32_t kv_encode4(float a, float b, float c, float d) {
  constexpr float Q = KvQmax<CODE>::value;
  a = a == a ? fminf(fmaxf(a, -Q), Q) : 0.0f;
  b = b == b ? fminf(fmaxf(b, -Q), Q) : 0.0f;
  c = c == c ? fminf(fmaxf(c, -Q), Q) : 0.0f;
  d = d == d ? fminf(fmaxf(d, -Q), Q) : 0.0f;
  if constexpr (CODE == IBP_KV_INT8) {
    constexpr float R = 12582912.0f;
    const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(a, R)),
                                    __float_as_uint(__fadd_rn(b, R)), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(c, R)),
                                    __float_as_uint(__fadd_rn(d, R)), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  } else {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
  }
}

// Four codes to the numbers they stand for (before the scale).
template <int CODE>
__device__ __forceinline__ void kv_decode4(uint32_t w, float *x) {
  if constexpr (CODE == IBP_KV_INT8) {
    // offset binary u = code + 128 in the low byte of 2^23's bit pattern
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)) - 8388736.0f;
  } else {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xFFFFu), __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
  }
}

// 16 consecutive elements of a row (16-byte aligned) as floats.
template <int DT>
__device__ __forceinline__ void load16(const void *p, float *x) {
  const uint4 *v = static_cast<const uint4 *>(p);
  if constexpr (DT == IBP_FP32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 w = __ldg(v + i);
      x[4 * i] = __uint_as_float(w.x);
      x[4 * i + 1] = __uint_as_float(w.y);
      x[4 * i + 2] = __uint_as_float(w.z);
      x[4 * i + 3] = __uint_as_float(w.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 w = __ldg(v + i);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (DT == IBP_BF16) {
          x[8 * i + 2 * k] = __uint_as_float(u[k] << 16);
          x[8 * i + 2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
        } else {
          const __half2 h = *reinterpret_cast<const __half2 *>(&u[k]);
          const float2 f = __half22float2(h);
          x[8 * i + 2 * k] = f.x;
          x[8 * i + 2 * k + 1] = f.y;
        }
      }
    }
  }
}

// Two floats rounded once to a pair of 16-bit elements.
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (DT == IBP_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
}

template <int DT>
__device__ __forceinline__ void store16(void *p, const float *x) {
  uint4 *v = static_cast<uint4 *>(p);
  if constexpr (DT == IBP_FP32) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                        __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v[i] = make_uint4(pack2<DT>(x[8 * i], x[8 * i + 1]), pack2<DT>(x[8 * i + 2], x[8 * i + 3]),
                        pack2<DT>(x[8 * i + 4], x[8 * i + 5]), pack2<DT>(x[8 * i + 6], x[8 * i + 7]));
  }
}

// Largest of the block's values (every thread gets it); `sm`: 32 floats.
__device__ __forceinline__ float block_max(float v, float *sm) {
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  if (blockDim.x <= 32) return v;
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float m = sm[0];
  for (int w = 1; w < (int)(blockDim.x >> 5); ++w) m = fmaxf(m, sm[w]);
  return m;
}

}  // namespace ibp
