// Append to the 8-bit paged key/value cache with the position rotation applied on the way
// (declared in include/ibp.h).
#include <algorithm>
#include <type_traits>

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
//
// 8 prompts of 4,096 tokens, 32 heads of 128 bf16, alone: K and V 207 us (805 MB, 3.9 TB/s; the
// append without a rotation 150), queries 92 (537 MB, 5.8 TB/s; a plain copy 82).
constexpr int MAX_THREADS = 512;
constexpr int GROUPS = 2;  // units of a head that a thread holds (rotated: 16 floats each)
constexpr int TURN_THREADS = 256;
constexpr int FEW_WARPS = 4;

struct RotateArgs {
  ibp_kv_cache c;
  ibp_kv_rows r;
  ibp_kv_rotation t;
  ibp_kv_turned q;
  int64_t each, items_each, items;
  int64_t kv_blocks;   // blocks that append; those after them rotate queries
  int q_chunks;        // blocks that share the heads of a query row
  int kv_chunks;       // blocks that share the heads of a page, of K or V
  bool apart;          // queries are rotated in a launch of their own
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
__device__ __forceinline__ Raw16<DT> load_unit(const char *row, const Unit &u) {
  constexpr int ES = DT == IBP_FP32 ? 4 : 2, V = DT == IBP_FP32 ? 2 : 1;
  Raw16<DT> r;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    r.v[i] = __ldg(reinterpret_cast<const uint4 *>(row + u.a * ES) + i);
    r.v[V + i] = __ldg(reinterpret_cast<const uint4 *>(row + u.b * ES) + i);
  }
  return r;
}

// Cosines and sines of a unit's pairs, two to a register pair.
struct Angles {
  uint64_t c[4], s[4];
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
      g.c[i] = pair(z.x, z.z);
      g.s[i] = pair(z.y, z.w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 z[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = 8 * u + 2 * i + k;
        z[k] = __ldg(reinterpret_cast<const float2 *>(
            a.t.d_table + 2 * (position_of(a, row, place, a.t.axis[at]) * pairs + at)));
      }
      g.c[i] = pair(z[0].x, z[1].x);
      g.s[i] = pair(z[0].y, z[1].y);
    }
  }
  return g;
}

// Two pairs (x, y): products two at a time, sums one by one (a packed product and sum could
// become one operation with one rounding).
__device__ __forceinline__ void turn2(float &x0, float &y0, float &x1, float &y1, uint64_t c, uint64_t s) {
  const uint64_t x = pair(x0, x1), y = pair(y0, y1);
  const uint64_t xc = mul2(x, c), ys = mul2(y, s), yc = mul2(y, c), xs = mul2(x, s);
  x0 = __fsub_rn(low(xc), low(ys));
  x1 = __fsub_rn(high(xc), high(ys));
  y0 = __fadd_rn(low(yc), low(xs));
  y1 = __fadd_rn(high(yc), high(xs));
}
__device__ __forceinline__ void turn_unit(float *x, const Angles &g, bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn2(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], g.c[i], g.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) turn2(x[2 * i], x[8 + 2 * i], x[2 * i + 1], x[9 + 2 * i], g.c[i], g.s[i]);
  }
}

// The larger of m and the magnitudes of 16 values, NaN if one is.
__device__ __forceinline__ float largest16(float m, const float *x) {
#pragma unroll
  for (int i = 0; i < 16; i += 2)
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(x[i]), "f"(x[i + 1]));
  return m;
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

// ---- queries: a thread turns one unit of a row in the heads of its share. Bound by HBM where there
// are many; few are bound by what is looked up before their first load (offsets, length, position,
// angles, one after another).
template <int D, int DT>
__device__ __forceinline__ void turn_queries(const RotateArgs &a, int64_t block) {
  constexpr int GD = D / 16, ES = DT == IBP_FP32 ? 4 : 2;
  constexpr int KEPT = 255;  // offsets that are searched in shared memory
  __shared__ int32_t starts[KEPT + 1];
  const int64_t row = block / a.q_chunks * (blockDim.x / GD) + threadIdx.x / GD;
  const int chunk = (int)(block % a.q_chunks);
  const bool kept = a.r.d_cu && a.c.batch <= KEPT;
  if (kept) {
    for (int i = threadIdx.x; i <= a.c.batch; i += blockDim.x) starts[i] = __ldg(a.r.d_cu + i);
    __syncthreads();
  }
  if (row >= a.r.n_rows) return;
  const Unit u = unit_of<D>(a.t, threadIdx.x % GD);
  int64_t place = 0;
  int b;
  if (a.r.d_cu) {
    int lo = 0, hi = a.c.batch;  // the last sequence that does not begin after the row
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if ((kept ? starts[mid] : __ldg(a.r.d_cu + mid)) <= row) lo = mid; else hi = mid;
    }
    b = lo;
    const int64_t first = kept ? starts[b] : __ldg(a.r.d_cu + b), end = kept ? starts[b + 1] : __ldg(a.r.d_cu + b + 1);
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
    const Raw16<DT> r = load_unit<DT>(from + h * a.q.q_head_stride * ES, u);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.four(i, x + 4 * i);
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

// Rows on their way: a thread copies its own units of the next heads into places of its own in
// shared memory, so that they wait for no barrier and take no registers.
template <int DT>
struct Ahead {
  static constexpr int vecs = Raw16<DT>::vecs, thread_bytes = GROUPS * vecs * 16;
  static constexpr int stages = DT == IBP_FP32 ? 3 : 4;  // heads, the one at hand among them
};
__device__ __forceinline__ void copy16(uint4 *to, const void *from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// Largest of the block's values; every thread gets it. `sm`: a place for each warp.
__device__ __forceinline__ uint32_t largest_of_block(uint32_t v, uint32_t *sm) {
  v = __reduce_max_sync(FULL, v);
  const int lane = threadIdx.x & 31;
  if (lane == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(FULL, lane < (int)(blockDim.x >> 5) ? sm[lane] : 0u);
}

// One thread block quantises what a page receives in some heads of K or V, one head after
// another: what follows from the place alone (sequence, page, the angles of its tokens) is worked
// out once for all of them, the next head's rows are asked for before this one's are rounded,
// and the values stay in registers between the maximum and the rounding, keys as rotated. (A head
// to a block took 342 us for what this takes 207.)
// Bound by the chain of a head: rows from shared memory, rotation, the block's maximum, codes;
// 16 warps an SM for the registers that rotated values and angles take (1.3 instructions a cycle,
// HBM 38 % busy). 80 registers and 24 warps spill (239 us), one unit a thread in blocks of 512
// takes 244, K and V in kernels of their own take as long as together.
// PLAIN: the rows fill the page, and keys are rotated whole in halves, so that nothing is asked
// for each unit (25 % fewer instructions).
template <int D, int DT, int CODE, bool KEYS, bool PLAIN>
__device__ __forceinline__ void append_heads(const RotateArgs &a, const AppendPlace &p, int h0, int h1,
                                             uint32_t (*sm)[32]) {
  constexpr int GD = D / 16, ES = DT == IBP_FP32 ? 4 : 2, HELD = KEYS ? IBP_FP32 : DT;
  using Held = Raw16<HELD>;
  using A = Ahead<DT>;
  extern __shared__ uint4 rows[];  // [stage][group][16 bytes][thread]
  const int P = 1 << a.shift, T = blockDim.x, STEP = T / GD;
  const int64_t row_stride = (KEYS ? a.r.k_row_stride : a.r.v_row_stride) * ES;
  const int64_t head_stride = (KEYS ? a.r.k_head_stride : a.r.v_head_stride) * ES;
  float *scale_at = (KEYS ? a.c.k_scales : a.c.v_scales) + (int64_t)p.page * a.c.n_heads + h0;
  char *codes = static_cast<char *>(KEYS ? a.c.k_codes : a.c.v_codes) + kv_tile(a.c, p.page, h0);
  // tokens of the tile: [old, fresh) are the new rows
  const int old = PLAIN ? 0 : (int)max((int64_t)p.len - p.t0, (int64_t)0);
  const int fresh = (int)min(p.end - p.t0, (int64_t)P);
  const int tok = threadIdx.x / GD, piece = threadIdx.x % GD;
  const Unit u = KEYS ? unit_of<D>(a.t, piece) : Unit{piece, 16 * piece, 16 * piece + 8, false};
  const int64_t row0 = p.lo + (p.t0 - p.len) + tok;
  const char *src = static_cast<const char *>(KEYS ? a.r.k : a.r.v) + row0 * row_stride + h0 * head_stride;
  const int64_t step = STEP * row_stride;
  auto live = [&](int i) { return PLAIN || (tok + i * STEP >= old && tok + i * STEP < fresh); };
  const int stage = GROUPS * A::vecs * T;
  uint4 *const first = rows + threadIdx.x, *const past = first + A::stages * stage;
  uint4 *to = first;
  int asked = h0;
  auto ask = [&] {  // for the next head's rows
    if (asked < h1) {
#pragma unroll
      for (int i = 0; i < GROUPS; ++i)
        if (live(i)) {
#pragma unroll
          for (int k = 0; k < A::vecs; ++k)
            copy16(to + (i * A::vecs + k) * T,
                   src + i * step + (k < A::vecs / 2 ? u.a * ES + 16 * k : u.b * ES + 16 * (k - A::vecs / 2)));
        }
      src += head_stride;
      ++asked;
      to += stage;
      if (to == past) to = first;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int k = 1; k < A::stages; ++k) ask();
  Angles g[KEYS ? GROUPS : 1];
  if constexpr (KEYS) {
#pragma unroll
    for (int i = 0; i < GROUPS; ++i)
      if (live(i) && u.turned) g[i] = angles_of(a, u.u, row0 + i * STEP, p.t0 + tok + i * STEP);
  }
  const uint4 *at = first;
  float next_before = old ? *scale_at : 0.0f;
  char *put_a = codes + tok * D + u.a, *put_b = codes + tok * D + u.b;
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const float before = next_before;
    cp_async_wait<A::stages - 2>();  // this head's rows (a thread reads none but its own copies)
    Raw16<DT> r[GROUPS];
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
      if constexpr (!PLAIN) r[i].clear();
      if (live(i))
#pragma unroll
        for (int k = 0; k < A::vecs; ++k) r[i].v[k] = at[(i * A::vecs + k) * T];
    }
    at += stage;
    if (at == past) at = first;
    Held x[GROUPS];
    uint32_t bits = 0;
    if constexpr (KEYS) {
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) {
        float y[16];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[i].four(e, y + 4 * e);
        if (PLAIN || (live(i) && u.turned)) turn_unit(y, g[i], !PLAIN && a.t.interleaved);
        most = largest16(most, y);
        x[i] = as_raw(y);
      }
      bits = __float_as_uint(most);
    } else {
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) {
        x[i] = r[i];
        bits = x[i].largest(bits);
      }
      bits = Held::fold(bits);
    }
    ask();
    if (old && h + 1 < h1) next_before = scale_at[1];
    // (two places in turn: a thread may be one barrier ahead of one that still reads)
    bits = largest_of_block(bits, sm[h & 1]);
    float largest = Held::value(bits);
    const bool odd = bits >= Held::inf;  // infinities or NaN among the values
    if (odd) {
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < GROUPS; ++i) most = largest_finite<HELD>(x[i], most);
      __syncthreads();
      largest = __uint_as_float(largest_of_block(__float_as_uint(most), sm[h & 1]));
    }
    const float scale = fmaxf(before, kv_scale<CODE>(largest));
    const float inverse = scale > 0.0f ? __frcp_rn(scale) : 0.0f;
    if (threadIdx.x == 0) *scale_at = scale;
    ++scale_at;
    auto put = [&](auto any) {
#pragma unroll
      for (int i = 0; i < GROUPS; ++i)
        if (live(i)) {
          const uint4 w = encode16<HELD, CODE, decltype(any)::value>(x[i], inverse);
          if constexpr (KEYS) {
            *reinterpret_cast<uint2 *>(put_a + i * STEP * D) = make_uint2(w.x, w.y);
            *reinterpret_cast<uint2 *>(put_b + i * STEP * D) = make_uint2(w.z, w.w);
          } else {
            *reinterpret_cast<uint4 *>(put_a + i * STEP * D) = w;
          }
        }
    };
    if (!odd && scale < 0x1p120f)
      put(std::false_type());
    else
      put(std::true_type());
    if (old && scale > before) {
      const float ratio = __fdiv_rn(before, scale);
      uint4 *there = reinterpret_cast<uint4 *>(codes) + threadIdx.x;
      for (int i = 0; tok + i * STEP < old; ++i) there[i * T] = rescale16<CODE>(there[i * T], ratio);
    }
    if constexpr (!PLAIN) codes += P * D;
    put_a += P * D;
    put_b += P * D;
  }
}

// Rows that queries are rotated in, after (and along with the end of) the kernel that appends.
template <int D, int DT>
__global__ void __launch_bounds__(TURN_THREADS, 4) kv_turn_kernel(const __grid_constant__ RotateArgs a) {
  turn_queries<D, DT>(a, blockIdx.x);
  grid_dependency_wait();  // what comes next in the stream may be ordered behind this grid alone
}

template <int D, int DT, int CODE>
__global__ void __launch_bounds__(MAX_THREADS)
    kv_rotate_kernel(const __grid_constant__ RotateArgs a) {
  __shared__ uint32_t sm[2][32];
  // For the queries' kernel, which reads nothing that this one writes. No other starts before this
  // one ends: it could hold an old line of scales in its first-level cache, which a block of this
  // one read for its own head while another's was still to be written.
  if (a.apart) grid_launch_dependents();
  if ((int64_t)blockIdx.x >= a.kv_blocks) {
    turn_queries<D, DT>(a, (int64_t)blockIdx.x - a.kv_blocks);
    return;
  }
  const int T = blockDim.x;
  const int64_t item = blockIdx.x / (2 * a.kv_chunks);
  const int which = (int)(blockIdx.x % (2 * a.kv_chunks)), chunk = which >> 1;
  Item i;
  if (a.r.d_cu) {
    int below = 0;  // starts rise with b: the last one that is not past the item
    for (int k0 = 0; k0 < a.c.batch; k0 += T) {
      const int k = k0 + (int)threadIdx.x;
      below += __syncthreads_count(k < a.c.batch && first_item(a.r, k, ShiftedPage{a.shift}) <= item);
    }
    i.b = max(below - 1, 0);
    i.nth = item - first_item(a.r, i.b, ShiftedPage{a.shift});
  } else {
    i = even_item(a, item);
  }
  const AppendPlace p = place_of(a.c, a.r, a.each, i.b, i.nth, ShiftedPage{a.shift}, which == 0 && threadIdx.x == 0,
                                 a.new_lens, a.status);
  if (p.page < 0) return;
  const int per = (a.c.n_heads + a.kv_chunks - 1) / a.kv_chunks, h0 = chunk * per,
            h1 = min(h0 + per, a.c.n_heads);
  if (h0 >= h1) return;
  const bool full = p.t0 >= p.len && p.end - p.t0 >= 1 << a.shift;
  if (which & 1) {
    if (full)
      append_heads<D, DT, CODE, false, true>(a, p, h0, h1, sm);
    else
      append_heads<D, DT, CODE, false, false>(a, p, h0, h1, sm);
  } else {
    if (full && a.t.dim == D && !a.t.interleaved)
      append_heads<D, DT, CODE, true, true>(a, p, h0, h1, sm);
    else
      append_heads<D, DT, CODE, true, false>(a, p, h0, h1, sm);
  }
}

// The same for a few rows a sequence: one warp to a tile, which reads its rows twice (the
// second time from L1). Bound by its chain of loads and the launch: one token for each of 64
// sequences, 8 heads of 128 with 32 query heads, 8.4 us alone and cold.
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
      const Raw16<DT> r = load_unit<DT>(at, u);
#pragma unroll
      for (int e = 0; e < 4; ++e) r.four(e, y + 4 * e);
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
      below += __popc(__ballot_sync(FULL, k0 + lane < a.c.batch && first_item(a.r, k0 + lane, ShiftedPage{a.shift}) <= item));
    i.b = max(below - 1, 0);
    i.nth = item - first_item(a.r, i.b, ShiftedPage{a.shift});
  } else {
    i = even_item(a, item);
  }
  const AppendPlace p =
      place_of(a.c, a.r, a.each, i.b, i.nth, ShiftedPage{a.shift}, which == 0 && lane == 0, a.new_lens, a.status);
  if (p.page < 0) return;
  if (which & 1)
    append_few<D, DT, CODE, false>(a, p, head, lane);
  else
    append_few<D, DT, CODE, true>(a, p, head, lane);
}

// Blocks of `threads` that rotate queries: up to 16 heads to a thread (its angles are loaded
// once), fewer while no more than `most` blocks come of it (those that run at once).
int64_t query_blocks(RotateArgs &a, int threads, int64_t most) {
  if (!a.q.q || a.r.n_rows == 0) return 0;
  const int rows = threads / (a.c.head_dim / 16);
  const int64_t blocks = (a.r.n_rows + rows - 1) / rows;
  a.q_chunks = (int)std::min<int64_t>(std::max<int64_t>(most / blocks, (a.q.q_heads + 15) / 16),
                                      a.q.q_heads);
  return blocks * a.q_chunks;
}

template <int D, int DT>
int launch_code(RotateArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const int P = a.c.page_tokens;
  a.each = a.r.d_cu ? 0 : a.r.n_rows / a.c.batch;
  a.items_each = a.each > 0 ? (a.each - 1) / P + 2 : 1;
  a.items = a.r.d_cu ? a.r.n_rows / P + 2 * (int64_t)a.c.batch : a.items_each * a.c.batch;
  if (a.items > 0x7FFFFFFF) return IBP_ERR_UNSUPPORTED;
  const bool int8 = a.c.code == IBP_KV_INT8;
  // A warp to a tile while a sequence brings less than a quarter of a page (the rule of the
  // append without a rotation, for the same reasons).
  if (a.r.n_rows < (int64_t)a.c.batch * (P / 4)) {
    constexpr int threads = 32 * FEW_WARPS;
    a.kv_blocks = (a.items * 2 * a.c.n_heads + FEW_WARPS - 1) / FEW_WARPS;
    const int64_t blocks = a.kv_blocks + query_blocks(a, threads, dev.sm_count);
    if (blocks > 0x7FFFFFFF) return IBP_ERR_UNSUPPORTED;
    const auto kernel = int8 ? kv_rotate_few_kernel<D, DT, IBP_KV_INT8> : kv_rotate_few_kernel<D, DT, IBP_KV_E4M3>;
    kernel<<<(unsigned)blocks, threads, 0, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? IBP_OK : IBP_ERR_CUDA;
  }
  const int threads = P * D / 16 / GROUPS;  // that hold a page: 32 (16 tokens of 64 elements) to 512
  // Up to 16 heads to a block (8 x 4,096 tokens, 32 heads of 128: 215 us with 8, 207 with 16,
  // 211 with 32). What a block looks up before its first row arrives takes as long as several
  // heads, so no more blocks than run at once where there are few pages.
  const int64_t at_once = (int64_t)dev.sm_count * std::min(512 / threads, 32);
  a.kv_chunks = (int)std::min<int64_t>(std::max<int64_t>(at_once / (a.items * 2), (a.c.n_heads + 15) / 16),
                                       a.c.n_heads);
  a.kv_blocks = a.items * 2 * a.kv_chunks;
  // Few queries along in the same launch; many in one of their own, which has half the registers
  // (whole calls with the read back: 3,500 rows of 8 heads of 64, 7 MB, 24.6 us | 26.7 in a launch of
  // their own; 5,556 rows of 28 heads of 128, 40 MB, 48 | 39).
  const bool apart = a.apart = a.q.q && a.r.n_rows * a.q.q_heads * D * (DT == IBP_FP32 ? 4 : 2) > (int64_t)(16 << 20);
  const int64_t turns = query_blocks(a, apart ? TURN_THREADS : threads, (apart ? 4 : 16) * (int64_t)dev.sm_count);
  const int64_t blocks = a.kv_blocks + (apart ? 0 : turns);
  if (blocks > 0x7FFFFFFF || turns > 0x7FFFFFFF) return IBP_ERR_UNSUPPORTED;
  const auto kernel = int8 ? kv_rotate_kernel<D, DT, IBP_KV_INT8> : kv_rotate_kernel<D, DT, IBP_KV_E4M3>;
  const int smem = threads * Ahead<DT>::thread_bytes * Ahead<DT>::stages;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return IBP_ERR_CUDA;
  kernel<<<(unsigned)blocks, threads, smem, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return IBP_ERR_CUDA;
  if (apart && turns > 0 && launch_dependent(kv_turn_kernel<D, DT>, dim3((unsigned)turns), dim3(TURN_THREADS), 0, s, a) != cudaSuccess)
    return IBP_ERR_CUDA;
  return IBP_OK;
}

template <int D>
int launch_dtype(RotateArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  switch (a.r.dtype) {
    case IBP_FP32: return launch_code<D, IBP_FP32>(a, dev, s);
    case IBP_FP16: return launch_code<D, IBP_FP16>(a, dev, s);
    default: return launch_code<D, IBP_BF16>(a, dev, s);
  }
}

}  // namespace

int launch_kv_append_rotated(const ibp_kv_cache &c, const ibp_kv_rows &r, const ibp_kv_rotation &t,
                             const ibp_kv_turned *q, int32_t *d_new_lens, int32_t *d_status,
                             cudaStream_t s) {
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
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
  return c.head_dim == 64 ? launch_dtype<64>(a, dev, s) : launch_dtype<128>(a, dev, s);
}

}  // namespace ibp
