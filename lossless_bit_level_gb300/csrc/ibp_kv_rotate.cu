// Append to the 8-bit paged key/value cache with the position rotation applied on the way
// (declared in include/ibp.h).
#include "ibp_kv_append.cuh"

namespace ibp {

namespace {

// Pair i of a head's first dim elements at position p: (x, y) -> (x c - y s, y c + x s) with
// (c, s) = table[p][i], every product and sum rounded once (never a fused multiply-add), so
// that equal inputs give equal codes. Keys are quantised from the rotated 32-bit values.
//
// A unit is 16 elements of a head in two pieces of 8: those that a unit's eight pairs (8 u to
// 8 u + 7) lie in. Pairs of two halves have pieces dim/2 apart, neighbouring pairs and what
// is not rotated lie in 16 consecutive elements.
constexpr int GROUPS = 4;       // units a thread holds (rotated: 16 floats each)
constexpr int MAX_THREADS = 256;  // a page of 128 tokens of 128 elements
constexpr int FEW_WARPS = 4;

struct RotateArgs {
  ibp_kv_cache c;
  ibp_kv_rows r;
  ibp_kv_rotation t;
  ibp_kv_turned q;
  int64_t each, items_each, items;
  int64_t kv_blocks;   // blocks that append; those after them rotate queries
  int q_chunks;        // blocks that share the heads of a query row
  int mixed;           // a unit's pairs are not all on one axis
  int shift;           // log2 of the page size
  int32_t *new_lens, *status;
};

struct Unit {
  int u, a, b;    // its number, first elements of its two pieces
  bool turned;
};
template <int D>
__device__ __forceinline__ Unit unit_of(const ibp_kv_rotation &t, int u) {
  Unit y;
  y.u = u;
  y.turned = 16 * u < t.dim;
  y.a = 16 * u;
  y.b = y.a + 8;
  if (y.turned && !t.interleaved) {
    y.a = 8 * u;
    y.b = y.a + t.dim / 2;
  }
  return y;
}

template <int DT>
__device__ __forceinline__ void load_unit(const char *row, const Unit &u, float *x) {
  constexpr int ES = DT == IBP_FP32 ? 4 : 2, V = DT == IBP_FP32 ? 2 : 1;
  Raw16<DT> r;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    r.v[i] = __ldg(reinterpret_cast<const uint4 *>(row + u.a * ES) + i);
    r.v[V + i] = __ldg(reinterpret_cast<const uint4 *>(row + u.b * ES) + i);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) r.four(i, x + 4 * i);
}

// Cosines and sines of a unit's pairs.
struct Angles {
  float2 y[8];
};
// Position of a row on an axis; `place`: its token's number in the sequence.
__device__ __forceinline__ int64_t position_of(const RotateArgs &a, int64_t row, int64_t place, int axis) {
  int64_t p = a.t.d_positions ? __ldg(a.t.d_positions + row * a.t.axes + axis) : place;
  const int64_t held = min(max(p, (int64_t)0), a.t.n_positions - 1);
  if (held != p) report(a.status, IBP_ERR_INDEX);
  return held;
}
__device__ __forceinline__ Angles angles_of(const RotateArgs &a, int u, int64_t row, int64_t place) {
  Angles g;
  const int pairs = a.t.dim / 2;
  if (!a.mixed) {
    const float4 *from = reinterpret_cast<const float4 *>(
        a.t.d_table + 2 * (position_of(a, row, place, a.t.axis[8 * u]) * pairs + 8 * u));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 z = __ldg(from + i);
      g.y[2 * i] = make_float2(z.x, z.y);
      g.y[2 * i + 1] = make_float2(z.z, z.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      g.y[i] = __ldg(reinterpret_cast<const float2 *>(
          a.t.d_table + 2 * (position_of(a, row, place, a.t.axis[8 * u + i]) * pairs + 8 * u + i)));
  }
  return g;
}

__device__ __forceinline__ void turn(float &x, float &y, float2 g) {
  const float u = __fsub_rn(__fmul_rn(x, g.x), __fmul_rn(y, g.y));
  y = __fadd_rn(__fmul_rn(y, g.x), __fmul_rn(x, g.y));
  x = u;
}
__device__ __forceinline__ void turn_unit(float *x, const Angles &g, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(x[2 * i], x[2 * i + 1], g.y[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(x[i], x[8 + i], g.y[i]);
  }
}

__device__ __forceinline__ Raw16<IBP_FP32> as_raw(const float *x) {
  Raw16<IBP_FP32> r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.v[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                        __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
  return r;
}

// The sequence of a work item, and which of its pages.
struct Item {
  int b;
  int64_t nth;
};
__device__ __forceinline__ Item even_item(const RotateArgs &a, int64_t item) {
  const int b = (int)(item / a.items_each);
  return {b, item - a.items_each * b};
}

// ---- queries: a thread turns one unit of a row in the heads of its share
template <int D, int DT>
__device__ __forceinline__ void turn_queries(const RotateArgs &a, int64_t block) {
  constexpr int GD = D / 16, ES = DT == IBP_FP32 ? 4 : 2;
  const int64_t row = block / a.q_chunks * (blockDim.x / GD) + threadIdx.x / GD;
  const int chunk = (int)(block % a.q_chunks);
  if (row >= a.r.n_rows) return;
  const Unit u = unit_of<D>(a.t, threadIdx.x % GD);
  int64_t place = 0;
  int b;
  if (a.r.d_cu) {
    int lo = 0, hi = a.c.batch;  // the last sequence that does not begin after the row
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (__ldg(a.r.d_cu + mid) <= row) lo = mid; else hi = mid;
    }
    b = lo;
    const int64_t first = __ldg(a.r.d_cu + b), end = __ldg(a.r.d_cu + b + 1);
    if (row < first || row >= end) return;  // no sequence's row
    place = row - first;
  } else {
    b = (int)(row / a.each);
    place = row - a.each * b;
  }
  Angles g;
  if (u.turned) {
    place += kv_len(a.c, b, a.status);
    g = angles_of(a, u.u, row, place);
  }
  const int per = (a.q.q_heads + a.q_chunks - 1) / a.q_chunks, h0 = chunk * per,
            h1 = min(h0 + per, a.q.q_heads);
  const char *from = static_cast<const char *>(a.q.q) + row * a.q.q_row_stride * ES;
  char *to = static_cast<char *>(a.q.out) + row * a.q.out_row_stride * ES;
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    float x[16];
    load_unit<DT>(from + h * a.q.q_head_stride * ES, u, x);
    if (u.turned) turn_unit(x, g, a.t.interleaved);
    char *out = to + h * a.q.out_head_stride * ES;
    if constexpr (DT == IBP_FP32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        reinterpret_cast<float4 *>(out + u.a * ES)[i] =
            make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        reinterpret_cast<float4 *>(out + u.b * ES)[i] =
            make_float4(x[8 + 4 * i], x[9 + 4 * i], x[10 + 4 * i], x[11 + 4 * i]);
      }
    } else {
      *reinterpret_cast<uint4 *>(out + u.a * ES) =
          make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7]));
      *reinterpret_cast<uint4 *>(out + u.b * ES) =
          make_uint4(pack2<DT>(x[8], x[9]), pack2<DT>(x[10], x[11]), pack2<DT>(x[12], x[13]),
                     pack2<DT>(x[14], x[15]));
    }
  }
}

// One thread block quantises what one (page, head) tile receives, as in the append without a
// rotation; the values stay in registers between the maximum and the rounding, keys as rotated.
template <int D, int DT, int CODE, bool KEYS>
__device__ __forceinline__ void append_tile(const RotateArgs &a, const AppendPlace &p, int head,
                                            uint32_t *sm) {
  constexpr int GD = D / 16, ES = DT == IBP_FP32 ? 4 : 2, HELD = KEYS ? IBP_FP32 : DT;
  const int P = 1 << a.shift, T = blockDim.x, STEP = T / GD;
  const int64_t row_stride = KEYS ? a.r.k_row_stride : a.r.v_row_stride;
  const int64_t head_stride = KEYS ? a.r.k_head_stride : a.r.v_head_stride;
  float *scale_at = (KEYS ? a.c.k_scales : a.c.v_scales) + (int64_t)p.page * a.c.n_heads + head;
  char *codes = static_cast<char *>(KEYS ? a.c.k_codes : a.c.v_codes) + kv_tile(a.c, p.page, head);
  const float before = p.t0 < p.len ? *scale_at : 0.0f;
  // tokens of the tile: [old, fresh) are the new rows
  const int old = (int)max((int64_t)p.len - p.t0, (int64_t)0), fresh = (int)min(p.end - p.t0, (int64_t)P);
  const int tok = threadIdx.x / GD;
  const Unit u = KEYS ? unit_of<D>(a.t, threadIdx.x % GD)
                      : Unit{(int)threadIdx.x % GD, 16 * ((int)threadIdx.x % GD), 0, false};
  const int64_t row0 = p.lo + (p.t0 - p.len) + tok;
  const char *src = static_cast<const char *>(KEYS ? a.r.k : a.r.v) +
                    (row0 * row_stride + head * head_stride) * ES;
  Raw16<HELD> x[GROUPS];
  uint32_t bits = 0;
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    x[g].clear();
    const int t = tok + g * STEP;
    if (t >= old && t < fresh) {
      const char *at = src + (int64_t)g * STEP * row_stride * ES;
      if constexpr (KEYS) {
        float y[16];
        load_unit<DT>(at, u, y);
        if (u.turned) turn_unit(y, angles_of(a, u.u, row0 + g * STEP, p.t0 + t), a.t.interleaved);
        x[g] = as_raw(y);
      } else {
        x[g].load(at + u.a * ES);
      }
    }
  }
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) bits = x[g].largest(bits);
  bits = block_max(Raw16<HELD>::fold(bits), sm);
  float largest = Raw16<HELD>::value(bits);
  const bool odd = bits >= Raw16<HELD>::inf;  // infinities or NaN among the values
  if (odd) {
    float most = 0.0f;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) most = largest_finite<HELD>(x[g], most);
    __syncthreads();
    largest = __uint_as_float(block_max(__float_as_uint(most), sm));
  }
  const float scale = fmaxf(before, kv_scale<CODE>(largest));
  const float inverse = kv_inverse(scale);
  if (threadIdx.x == 0) *scale_at = scale;
  const bool any = odd || !(scale < 0x1p120f);
#pragma unroll
  for (int g = 0; g < GROUPS; ++g) {
    const int t = tok + g * STEP;
    if (t >= old && t < fresh) {
      const uint4 w = any ? encode16<HELD, CODE, true>(x[g], inverse) : encode16<HELD, CODE, false>(x[g], inverse);
      char *to = codes + t * D;
      if constexpr (KEYS) {
        *reinterpret_cast<uint2 *>(to + u.a) = make_uint2(w.x, w.y);
        *reinterpret_cast<uint2 *>(to + u.b) = make_uint2(w.z, w.w);
      } else {
        *reinterpret_cast<uint4 *>(to + u.a) = w;
      }
    }
  }
  if (old && scale > before) {
    const float ratio = __fdiv_rn(before, scale);
    uint4 *there = reinterpret_cast<uint4 *>(codes) + threadIdx.x;
    for (int g = 0; tok + g * STEP < old; ++g) there[g * T] = rescale16<CODE>(there[g * T], ratio);
  }
}

template <int D, int DT, int CODE>
__global__ void __launch_bounds__(MAX_THREADS) kv_rotate_kernel(const __grid_constant__ RotateArgs a) {
  __shared__ uint32_t sm[32];
  if ((int64_t)blockIdx.x >= a.kv_blocks) {
    turn_queries<D, DT>(a, (int64_t)blockIdx.x - a.kv_blocks);
    return;
  }
  const int T = blockDim.x;
  const int64_t item = blockIdx.x / (2 * a.c.n_heads);
  const int which = (int)(blockIdx.x % (2 * a.c.n_heads)), head = which >> 1;
  Item i;
  if (a.r.d_cu) {
    int below = 0;  // starts rise with b: the last one that is not past the item
    for (int k0 = 0; k0 < a.c.batch; k0 += T) {
      const int k = k0 + (int)threadIdx.x;
      below += __syncthreads_count(k < a.c.batch && first_item(a.r, k, a.shift) <= item);
    }
    i.b = max(below - 1, 0);
    i.nth = item - first_item(a.r, i.b, a.shift);
  } else {
    i = even_item(a, item);
  }
  const AppendPlace p = place_of(a.c, a.r, a.each, i.b, i.nth, a.shift, which == 0 && threadIdx.x == 0,
                                 a.new_lens, a.status);
  if (p.page < 0) return;
  if (which & 1)
    append_tile<D, DT, CODE, false>(a, p, head, sm);
  else
    append_tile<D, DT, CODE, true>(a, p, head, sm);
}

// The same for a few rows a sequence: one warp to a tile, which reads its rows twice (the
// second time from L1).
template <int D, int DT, int CODE, bool KEYS>
__device__ __forceinline__ void append_few(const RotateArgs &a, const AppendPlace &p, int head, int lane) {
  constexpr int GD = D / 16, ES = DT == IBP_FP32 ? 4 : 2, HELD = KEYS ? IBP_FP32 : DT;
  const int64_t row_stride = KEYS ? a.r.k_row_stride : a.r.v_row_stride;
  const int64_t head_stride = KEYS ? a.r.k_head_stride : a.r.v_head_stride;
  float *scale_at = (KEYS ? a.c.k_scales : a.c.v_scales) + (int64_t)p.page * a.c.n_heads + head;
  char *codes = static_cast<char *>(KEYS ? a.c.k_codes : a.c.v_codes) + kv_tile(a.c, p.page, head);
  const float before = p.t0 < p.len ? *scale_at : 0.0f;
  const int64_t from = max(p.t0, (int64_t)p.len), to = min(p.end, p.t0 + (1 << a.shift));
  const int units = (int)(to - from) * GD, t0 = (int)(from - p.t0);
  const int64_t row0 = p.lo + (from - p.len);
  const char *src = static_cast<const char *>(KEYS ? a.r.k : a.r.v) + (row0 * row_stride + head * head_stride) * ES;
  const Unit u = KEYS ? unit_of<D>(a.t, lane % GD) : Unit{lane % GD, 16 * (lane % GD), 0, false};
  auto load = [&](int i) {
    Raw16<HELD> x;
    const char *at = src + (int64_t)(i / GD) * row_stride * ES;
    if constexpr (KEYS) {
      float y[16];
      load_unit<DT>(at, u, y);
      if (u.turned) turn_unit(y, angles_of(a, u.u, row0 + i / GD, from + i / GD), a.t.interleaved);
      x = as_raw(y);
    } else {
      x.load(at + u.a * ES);
    }
    return x;
  };
  uint32_t bits = 0;
  for (int i = lane; i < units; i += 32) bits = load(i).largest(bits);
  bits = __reduce_max_sync(FULL, Raw16<HELD>::fold(bits));
  float largest = Raw16<HELD>::value(bits);
  const bool odd = bits >= Raw16<HELD>::inf;
  if (odd) {
    float most = 0.0f;
    for (int i = lane; i < units; i += 32) most = largest_finite<HELD>(load(i), most);
    largest = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(most)));
  }
  const float scale = fmaxf(before, kv_scale<CODE>(largest));
  const float inverse = kv_inverse(scale);
  if (lane == 0) *scale_at = scale;
  const bool any = odd || !(scale < 0x1p120f);
  for (int i = lane; i < units; i += 32) {
    const Raw16<HELD> x = load(i);
    const uint4 w = any ? encode16<HELD, CODE, true>(x, inverse) : encode16<HELD, CODE, false>(x, inverse);
    char *out = codes + (t0 + i / GD) * D;
    if constexpr (KEYS) {
      *reinterpret_cast<uint2 *>(out + u.a) = make_uint2(w.x, w.y);
      *reinterpret_cast<uint2 *>(out + u.b) = make_uint2(w.z, w.w);
    } else {
      *reinterpret_cast<uint4 *>(out + u.a) = w;
    }
  }
  if (scale > before) {
    const float ratio = __fdiv_rn(before, scale);
    uint4 *there = reinterpret_cast<uint4 *>(codes);
    for (int i = lane; i < t0 * GD; i += 32) there[i] = rescale16<CODE>(there[i], ratio);
  }
}

template <int D, int DT, int CODE>
__global__ void __launch_bounds__(32 * FEW_WARPS) kv_rotate_few_kernel(const __grid_constant__ RotateArgs a) {
  if ((int64_t)blockIdx.x >= a.kv_blocks) {
    turn_queries<D, DT>(a, (int64_t)blockIdx.x - a.kv_blocks);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t warp = (int64_t)blockIdx.x * FEW_WARPS + (threadIdx.x >> 5);
  const int64_t item = warp / (2 * a.c.n_heads);
  const int which = (int)(warp % (2 * a.c.n_heads)), head = which >> 1;
  if (item >= a.items) return;
  Item i;
  if (a.r.d_cu) {
    int below = 0;
    for (int k0 = 0; k0 < a.c.batch; k0 += 32)
      below += __popc(__ballot_sync(FULL, k0 + lane < a.c.batch && first_item(a.r, k0 + lane, a.shift) <= item));
    i.b = max(below - 1, 0);
    i.nth = item - first_item(a.r, i.b, a.shift);
  } else {
    i = even_item(a, item);
  }
  const AppendPlace p =
      place_of(a.c, a.r, a.each, i.b, i.nth, a.shift, which == 0 && lane == 0, a.new_lens, a.status);
  if (p.page < 0) return;
  if (which & 1)
    append_few<D, DT, CODE, false>(a, p, head, lane);
  else
    append_few<D, DT, CODE, true>(a, p, head, lane);
}

// Blocks that rotate queries, `threads` each.
int64_t query_blocks(RotateArgs &a, int threads, int heads_each) {
  if (!a.q.q || a.r.n_rows == 0) return 0;
  const int rows = threads / (a.c.head_dim / 16);
  a.q_chunks = (a.q.q_heads + heads_each - 1) / heads_each;
  return (a.r.n_rows + rows - 1) / rows * a.q_chunks;
}

template <int D, int DT>
int launch_code(RotateArgs &a, cudaStream_t s) {
  const int P = a.c.page_tokens;
  a.each = a.r.d_cu ? 0 : a.r.n_rows / a.c.batch;
  a.items_each = a.each > 0 ? (a.each - 1) / P + 2 : 1;
  a.items = a.r.d_cu ? a.r.n_rows / P + 2 * (int64_t)a.c.batch : a.items_each * a.c.batch;
  const bool int8 = a.c.code == IBP_KV_INT8;
  // A warp to a tile while a sequence brings less than a quarter of a page (the rule of the
  // append without a rotation, for the same reasons).
  const bool few = a.r.n_rows < (int64_t)a.c.batch * (P / 4);
  const int threads = few ? 32 * FEW_WARPS : P * D / 16 / GROUPS < 32 ? 32 : P * D / 16 / GROUPS;
  a.kv_blocks = few ? (a.items * 2 * a.c.n_heads + FEW_WARPS - 1) / FEW_WARPS : a.items * 2 * a.c.n_heads;
  const int64_t blocks = a.kv_blocks + query_blocks(a, threads, few ? 4 : 8);
  if (a.items > 0x7FFFFFFF || blocks > 0x7FFFFFFF) return IBP_ERR_UNSUPPORTED;
  const auto kernel = few ? (int8 ? kv_rotate_few_kernel<D, DT, IBP_KV_INT8> : kv_rotate_few_kernel<D, DT, IBP_KV_E4M3>)
                          : (int8 ? kv_rotate_kernel<D, DT, IBP_KV_INT8> : kv_rotate_kernel<D, DT, IBP_KV_E4M3>);
  kernel<<<(unsigned)blocks, threads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? IBP_OK : IBP_ERR_CUDA;
}

template <int D>
int launch_dtype(RotateArgs &a, cudaStream_t s) {
  switch (a.r.dtype) {
    case IBP_FP32: return launch_code<D, IBP_FP32>(a, s);
    case IBP_FP16: return launch_code<D, IBP_FP16>(a, s);
    default: return launch_code<D, IBP_BF16>(a, s);
  }
}

}  // namespace

int launch_kv_append_rotated(const ibp_kv_cache &c, const ibp_kv_rows &r, const ibp_kv_rotation &t,
                             const ibp_kv_turned *q, int32_t *d_new_lens, int32_t *d_status,
                             cudaStream_t s) {
  RotateArgs a = {};
  a.c = c;
  a.r = r;
  a.t = t;
  if (q) a.q = *q;
  a.q_chunks = 1;
  a.shift = page_shift(c.page_tokens);
  for (int i = 0; i < t.dim / 2; ++i) a.mixed |= t.axis[i] != t.axis[i & ~7];
  a.new_lens = d_new_lens;
  a.status = d_status;
  return c.head_dim == 64 ? launch_dtype<64>(a, s) : launch_dtype<128>(a, s);
}

}  // namespace ibp
