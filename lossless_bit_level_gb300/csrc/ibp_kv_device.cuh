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

// How a CTA goes over one (page, head) tile: every thread holds `per_thread` groups of 16
// consecutive elements of a token. Eight groups a thread where that leaves a warp: what a
// thread works out once (its sequence, page, addresses, the tile's maximum) costs as much as
// converting 16 elements or two (moving 8 x 2,048 tokens, 32 heads of 128: 67 us with two
// groups a thread, 54 with four, 52 with eight).
template <int P, int D>
struct Tile {
  static constexpr int groups = P * D / 16;
  static constexpr int threads = groups < 256 ? 32 : groups / 8;
  static constexpr int per_thread = groups / threads;
  static constexpr int step = threads / (D / 16);  // tokens between a thread's groups
};

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

// Pairs of floats in one instruction, to spare issue slots. A packed product that goes into
// a packed sum may become one operation with one rounding: kept apart where codes depend
// on it (kv_encode4 adds one by one).
__device__ __forceinline__ uint64_t pair(float a, float b) {
  return (uint64_t)__float_as_uint(a) | ((uint64_t)__float_as_uint(b) << 32);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float low(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float high(uint64_t x) { return __uint_as_float((uint32_t)(x >> 32)); }
__device__ __forceinline__ void mul4(float *x, float f) {
  const uint64_t ff = pair(f, f), a = mul2(pair(x[0], x[1]), ff), b = mul2(pair(x[2], x[3]), ff);
  x[0] = low(a);
  x[1] = high(a);
  x[2] = low(b);
  x[3] = high(b);
}

// Four values (already times the inverse scale) to four codes in one word. int8:
// adding 1.5 * 2^23 leaves the value rounded to nearest even in the low byte (the magic-number
// conversion: Warren, Hacker's Delight, chapter on floating point). Values a
// rounding or two past +-qmax round to qmax; anything further, and NaN, needs
// kv_encode4_any.
template <int CODE>
__device__ __forceinline__ uint32_t kv_encode4(float a, float b, float c, float d) {
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
template <int CODE>
__device__ __forceinline__ float kv_saturate(float a) {
  constexpr float Q = KvQmax<CODE>::value;
  return a == a ? fminf(fmaxf(a, -Q), Q) : 0.0f;
}
template <int CODE>
__device__ __forceinline__ uint32_t kv_encode4_any(float a, float b, float c, float d) {
  return kv_encode4<CODE>(kv_saturate<CODE>(a), kv_saturate<CODE>(b), kv_saturate<CODE>(c),
                          kv_saturate<CODE>(d));
}

// Four codes to the numbers they stand for (before the scale).
template <int CODE>
__device__ __forceinline__ void kv_decode4(uint32_t w, float *x) {
  if constexpr (CODE == IBP_KV_INT8) {
    // offset binary u = code + 128 in the low byte of 2^23's bit pattern
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint64_t y = add2(pair(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)),
                                   __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441 + i))),
                              pair(-8388736.0f, -8388736.0f));
      x[i] = low(y);
      x[i + 1] = high(y);
    }
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

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}

__device__ __forceinline__ uint32_t max_s16x2(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.s16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
__device__ __forceinline__ uint32_t min_s16x2(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("min.s16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}

// 16 consecutive elements of a row (16-byte aligned) as they lie in memory.
template <int DT>
struct Raw16 {
  static constexpr int vecs = DT == IBP_FP32 ? 4 : 2;
  // magnitude bits of an infinity: everything finite lies below
  static constexpr uint32_t inf = DT == IBP_FP32 ? 0x7F800000u : DT == IBP_BF16 ? 0x7F80u : 0x7C00u;
  uint4 v[vecs];
  __device__ __forceinline__ void load(const void *p) {
#pragma unroll
    for (int i = 0; i < vecs; ++i) v[i] = __ldg(static_cast<const uint4 *>(p) + i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < vecs; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4 w = v[i / 4];
    return i % 4 == 0 ? w.x : i % 4 == 1 ? w.y : i % 4 == 2 ? w.z : w.w;
  }
  // Elements 4i .. 4i + 3 as floats.
  __device__ __forceinline__ void four(int i, float *x) const {
    if constexpr (DT == IBP_FP32) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = __uint_as_float(word(4 * i + k));
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t u = word(2 * i + k);
        if constexpr (DT == IBP_BF16) {
          x[2 * k] = __uint_as_float(u << 16);
          x[2 * k + 1] = __uint_as_float(u & 0xFFFF0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
          x[2 * k] = f.x;
          x[2 * k + 1] = f.y;
        }
      }
    }
  }
  // The larger of m and the elements' magnitude bits (16-bit types: of both halves apart).
  __device__ __forceinline__ uint32_t largest(uint32_t m) const {
#pragma unroll
    for (int i = 0; i < 4 * vecs; ++i)
      m = DT == IBP_FP32 ? max(m, word(i) & 0x7FFFFFFFu) : max_u16x2(m, word(i) & 0x7FFF7FFFu);
    return m;
  }
  __device__ __forceinline__ static uint32_t fold(uint32_t m) {
    return DT == IBP_FP32 ? m : max(m >> 16, m & 0xFFFFu);
  }
  __device__ __forceinline__ static float value(uint32_t bits) {
    return DT == IBP_FP32   ? __uint_as_float(bits)
           : DT == IBP_BF16 ? __uint_as_float(bits << 16)
                            : __half2float(__ushort_as_half((unsigned short)bits));
  }
};

template <int DT>
__device__ __forceinline__ void load16(const void *p, float *x) {
  Raw16<DT> r;
  r.load(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) r.four(i, x + 4 * i);
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

// Largest of the block's values (every thread gets it); `sm`: 32 words.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *sm) {
  v = __reduce_max_sync(FULL, v);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t m = sm[0];
  for (int w = 1; w < (int)(blockDim.x >> 5); ++w) m = max(m, sm[w]);
  return m;
}

}  // namespace ibp
