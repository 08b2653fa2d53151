// Selecting pages of the 8-bit paged key/value cache for each sequence and K/V head by a cheap
// score (declared in include/ibp.h): bounds of each page's key codes, the score of a page, and
// the columns of the highest.
#include <algorithm>

#include "ibp_kv_attention.cuh"

namespace ibp {

namespace {

constexpr int SLAB_BATCH = 1024;  // sequences of one launch (their item counts are in shared memory)

// Items before each of n sequences, prefix[n] of them in all (one warp; count(b) >= 0).
template <typename F>
__device__ __forceinline__ void count_items(int64_t *prefix, int n, F count) {
  const int lane = threadIdx.x & 31;
  int64_t base = 0;
  for (int k0 = 0; k0 < n; k0 += 32) {
    const int b = k0 + lane;
    const int64_t mine = b < n ? count(b) : 0;
    int64_t sum = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(FULL, sum, o);
      if (lane >= o) sum += y;
    }
    if (b < n) prefix[b] = base + sum - mine;
    base += __shfl_sync(FULL, sum, 31);
  }
  if (lane == 0) prefix[n] = base;
}

// ---- bounds ------------------------------------------------------------------------

struct BoundsArgs {
  ibp_kv_cache c;
  int8_t *bounds;
  const int32_t *begin;
  int32_t *status;
  int b0, batch;
};

// Codes as bytes in the order of their numbers: int8 as they are, e4m3 (sign and magnitude)
// with the magnitude bits of negative ones turned over. The same again turns them back.
template <int CODE>
__device__ __forceinline__ uint32_t in_order(uint32_t w) {
  if constexpr (CODE == IBP_KV_INT8) return w;
  const uint32_t sign = w & 0x80808080u;
  return w ^ (sign - (sign >> 7));
}

// A bound in whole units: int8 codes as they are; e4m3 numbers in units of 448/127, rounded down
// (the least) or up (the largest). c * 127 / 448 is whole at 0 and +-448 only, and elsewhere
// far from whole against the rounding of the division.
template <int CODE>
__device__ __forceinline__ int bound_unit(uint32_t byte, bool up) {
  if constexpr (CODE == IBP_KV_INT8) return max((int)(int8_t)byte, -127);
  const uint32_t magnitude = min(byte & 0x7Fu, 0x7Eu);  // (a NaN as the largest of its sign)
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)((byte & 0x80u) | magnitude), __NV_E4M3);
  const float x = __fdiv_rn(__half2float(__half(h)) * 127.0f, 448.0f);
  return (int)(up ? ceilf(x) : floorf(x));
}

constexpr int BOUNDS_THREADS = 256;

// Least and largest code of each element over a tile's tokens. One warp to a (page, head) tile:
// a lane takes 16 elements of every 32/(D/16)-th token and keeps least and largest as pairs of
// bytes in the upper halves of 16-bit lanes (what lies below a byte there is cleared), then the
// lanes of the same elements exchange theirs. Bound by HBM: every code is read once, eight loads
// a lane at a time, and the next tile's page is looked up before this one's codes are there.
// 8 sequences of 4,096 tokens, 32 heads of 128 (138 MB): 26 us, 5.3 TB/s (four loads at a time, the
// page looked up first: 31).
template <int D, int CODE>
__global__ void __launch_bounds__(BOUNDS_THREADS, 3) kv_bounds_kernel(const __grid_constant__ BoundsArgs a) {
  constexpr int PIECES = D / 16, STEP = 32 / PIECES, AHEAD = 8;
  __shared__ int64_t prefix[SLAB_BATCH + 1];
  const ibp_kv_cache &c = a.c;
  const int P = c.page_tokens, lane = threadIdx.x & 31, piece = lane % PIECES;
  grid_launch_dependents();
  auto first_page = [&](int b) { return a.begin ? max(__ldg(a.begin + a.b0 + b), 0) / P : 0; };
  if (threadIdx.x < 32)
    count_items(prefix, a.batch, [&](int b) {
      const int pages = (kv_len(c, a.b0 + b, blockIdx.x == 0 ? a.status : nullptr) + P - 1) / P;
      return (int64_t)max(pages - first_page(b), 0) * c.n_heads;
    });
  __syncthreads();
  const int64_t total = prefix[a.batch], warps = (int64_t)gridDim.x * (BOUNDS_THREADS / 32);
  struct Tile {
    int page, head, held;
  };
  auto look_up = [&](int64_t x) {
    Tile t = {-1, 0, 0};
    if (x >= total) return t;
    const int b = find_sequence(prefix, a.batch, x);
    const int64_t in = x - prefix[b];
    const int j = (in >> 31) == 0 ? (int)((uint32_t)in / (uint32_t)c.n_heads) : (int)(in / c.n_heads);
    const int col = first_page(b) + j;
    t.head = (int)(in - (int64_t)j * c.n_heads);
    t.page = kv_page(c, a.b0 + b, col, a.status);
    t.held = min(kv_len(c, a.b0 + b, nullptr) - col * P, P);
    return t;
  };
  int64_t x = (int64_t)blockIdx.x * (BOUNDS_THREADS / 32) + (threadIdx.x >> 5);
  Tile next = look_up(x);
  for (; x < total; x += warps) {
    const Tile now = next;
    next = look_up(x + warps);
    if (now.page < 0) continue;
    const uint4 *codes = reinterpret_cast<const uint4 *>(static_cast<const char *>(c.k_codes) +
                                                         kv_tile(c, now.page, now.head)) + lane;
    uint32_t low[4][2], high[4][2];  // [word][bytes 0, 2 | 1, 3]
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        low[i][k] = 0x7F007F00u;
        high[i][k] = 0x80008000u;
      }
    for (int t = lane / PIECES; t < now.held; t += AHEAD * STEP, codes += AHEAD * 32) {
      uint4 v[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)  // (a token past the last: the lane's first again)
        v[k] = __ldg(codes + (t + k * STEP < now.held ? k * 32 : 0));
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t o = in_order<CODE>(w[i]), even = (o << 8) & 0xFF00FF00u, odd = o & 0xFF00FF00u;
          low[i][0] = min_s16x2(low[i][0], even);
          high[i][0] = max_s16x2(high[i][0], even);
          low[i][1] = min_s16x2(low[i][1], odd);
          high[i][1] = max_s16x2(high[i][1], odd);
        }
      }
    }
#pragma unroll
    for (int o = PIECES; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          low[i][k] = min_s16x2(low[i][k], __shfl_xor_sync(FULL, low[i][k], o));
          high[i][k] = max_s16x2(high[i][k], __shfl_xor_sync(FULL, high[i][k], o));
        }
    if (lane < 2 * PIECES) {  // the first PIECES lanes write the least, the next the largest
      const bool up = lane >= PIECES;
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t y = in_order<CODE>(up ? (high[i][0] >> 8) | high[i][1] : (low[i][0] >> 8) | low[i][1]);
        w[i] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          w[i] |= (uint32_t)(bound_unit<CODE>((y >> (8 * k)) & 0xFFu, up) & 0xFF) << (8 * k);
      }
      reinterpret_cast<uint4 *>(a.bounds + ((int64_t)now.page * c.n_heads + now.head) * 2 * D)[up * PIECES + piece] =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ---- score -------------------------------------------------------------------------

constexpr int SCORE_WARPS = 4, SCORE_THREADS = 32 * SCORE_WARPS;
constexpr int CHUNK = 16 * SCORE_WARPS;  // pages of an item: 16 a warp
constexpr int ROWS = 64;                 // query rows in shared memory at a time

struct SelectArgs {
  ibp_kv_cache c;
  ibp_kv_query q;
  const int8_t *bounds;
  float *scores;     // [batch][n_heads][table_cols]
  int32_t *columns;  // [batch][n_heads][pages]
  int32_t *status;
  int pages, b0, batch;
};

// The rows of a sequence: as attention counts them.
__device__ __forceinline__ int rows_at(const SelectArgs &a, int b, int64_t *row0, int32_t *status) {
  int64_t lo, hi;
  kv_row_range(a.q.d_cu, a.q.n_rows, a.q.max_q, b, status, &lo, &hi);
  if (hi - lo > a.q.max_q) {
    report(status, IBP_ERR_INDEX);
    hi = lo + a.q.max_q;
  }
  *row0 = lo;
  return (int)(hi - lo);
}

__device__ __forceinline__ void mma_f16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Bytes 0, 1 (HIGH = 0) or 2, 3 of a word of code + 128 as two fp16: the byte below 0x64 is
// 1024 + 128 + code.
template <int HIGH>
__device__ __forceinline__ uint32_t whole_pair(uint32_t u) {
  const uint32_t x = __byte_perm(u, 0x64646464u, HIGH ? 0x4342 : 0x4140);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Rows r0 .. r0 + some - 1 of a sequence and K/V head (in whole tiles of 8) in whole numbers, as the
// lanes hold the second operand: every warp takes some.
template <int D, int DT, bool ONE, int WARPS>
__device__ __forceinline__ void rows_in_whole_numbers(const SelectArgs &a, int64_t row0, int head, int r0, int some,
                                                      int tiles, uint2 (*rows)[D / 8][32], float *unit) {
  constexpr int STEPS = D / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = a.q.q_heads / a.c.n_heads;
          constexpr int BATCH = ONE ? 2 : 4;  // rows of a warp that are asked for at a time
          for (int r1 = warp; r1 < 8 * tiles; r1 += BATCH * WARPS) {
            uint2 asked[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
              const int r = r1 + k * WARPS, rr = r0 + r;
              asked[k] = make_uint2(0u, 0u);
              if (r < some && lane < D / 4)
                asked[k] = __ldg(reinterpret_cast<const uint2 *>(
                    static_cast<const char *>(a.q.q) + 2 * ((row0 + rr / group) * a.q.q_row_stride +
                                                            (head * group + rr % group) * a.q.q_head_stride + 4 * lane)));
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
              const int r = r1 + k * WARPS;
              if (r >= 8 * tiles) break;
              float q[4];
              const uint32_t words[2] = {asked[k].x, asked[k].y};
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if constexpr (DT == IBP_BF16) {
                  q[2 * i] = __uint_as_float(words[i] << 16);
                  q[2 * i + 1] = __uint_as_float(words[i] & 0xFFFF0000u);
                } else {
                  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&words[i]));
                  q[2 * i] = f.x;
                  q[2 * i + 1] = f.y;
                }
              }
              // (a NaN is not counted; where all four are, the 0 is what is left)
              float most = fmaxf(fmaxf(fmaxf(fabsf(q[0]), fabsf(q[1])), fmaxf(fabsf(q[2]), fabsf(q[3]))), 0.0f);
              most = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(most)));
              const int e = min(max((int)(__float_as_uint(most) >> 23) - 127, -100), 100);
              const float up = __uint_as_float((uint32_t)(127 + 6 - e) << 23);
              if (lane == 0)
                unit[r] = r < some ? __uint_as_float((uint32_t)(127 - 6 + e) << 23) : __uint_as_float(0x7FFFFFFFu);
              uint32_t w[2][2];
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                float y[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const float z = rintf(q[i + k] * up);
                  y[k] = z == z ? fminf(fmaxf(z, -127.0f), 127.0f) : 0.0f;
                }
                w[0][i / 2] = pack2<IBP_FP16>(fminf(y[0], 0.0f), fminf(y[1], 0.0f));
                w[1][i / 2] = pack2<IBP_FP16>(fmaxf(y[0], 0.0f), fmaxf(y[1], 0.0f));
              }
              if (lane < D / 4) {  // elements 4 lane ..: bytes 16 t + 4 e .. of 64 j
                const int j = lane / 16, t = lane % 16 / 4, step = 4 * j + lane % 4;
                rows[r / 8][step][(r % 8) * 4 + t] = make_uint2(w[0][0], w[0][1]);
                rows[r / 8][STEPS / 2 + step][(r % 8) * 4 + t] = make_uint2(w[1][0], w[1][1]);
              }
            }
          }
}

// 16 pages' bounds: lane (g, t) holds bytes 16 t .. of pages g and g + 8 (page < 0: none).
template <int D>
struct Pages16 {
  static constexpr int K = 2 * D, STEPS = K / 16;
  float scale[2];
  bool there[2];
  uint4 raw[2][K / 64];
  __device__ __forceinline__ void load(const SelectArgs &a, const int *page, int head) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      there[h] = page[h] >= 0;
      const int64_t tile = (int64_t)page[h] * a.c.n_heads + head;
      scale[h] = there[h] ? __ldg(a.c.k_scales + tile) : 0.0f;
#pragma unroll
      for (int j = 0; j < K / 64; ++j)
        raw[h][j] = there[h] ? __ldg(reinterpret_cast<const uint4 *>(a.bounds + tile * K) + (threadIdx.x & 3) + 4 * j)
                             : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void operand(int step, uint32_t *m) const {  // 16 bytes of both, as fp16
    const int j = step / 4, e = step % 4;
    const uint4 r = raw[0][j], q = raw[1][j];
    const uint32_t u = (e == 0 ? r.x : e == 1 ? r.y : e == 2 ? r.z : r.w) ^ 0x80808080u,
                   v = (e == 0 ? q.x : e == 1 ? q.y : e == 2 ? q.z : q.w) ^ 0x80808080u;
    m[0] = whole_pair<0>(u);
    m[1] = whole_pair<0>(v);
    m[2] = whole_pair<1>(u);
    m[3] = whole_pair<1>(v);
  }
  // the largest of best and the tiles' scores before the pages' scales
  template <bool ONE>
  __device__ __forceinline__ void against(float *best, const uint32_t (*m)[4], int tiles, const uint2 (*rows)[STEPS][32],
                                          const float *unit) const {
    const int lane = threadIdx.x & 31, t4 = lane & 3;
    for (int i = 0; i < tiles; ++i) {
      float even[4] = {}, odd[4] = {};  // two chains: a chain waits for each of its own
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        const uint2 y = rows[i][k][lane];
        uint32_t w[4];
        if constexpr (ONE) operand(k, w);
        const uint32_t *x = ONE ? w : m[ONE ? 0 : k];
        mma_f16(k & 1 ? odd : even, x[0], x[1], x[2], x[3], y.x, y.y);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        best[k >> 1] = fmaxf(best[k >> 1], (even[k] + odd[k]) * unit[8 * i + 2 * t4 + (k & 1)]);
    }
  }
  // over the lanes of a page, times its scale
  __device__ __forceinline__ float score(float best, int h) const {
    best = fmaxf(best, __shfl_xor_sync(FULL, best, 1));
    best = fmaxf(best, __shfl_xor_sync(FULL, best, 2));
    return there[h] ? __fmul_rn(best, scale[h]) : -INFINITY;
  }
};

// score = scale_k max_r 2^(e_r - 6) sum_d max(n_rd least_d, n_rd largest_d), with the query row
// r in whole numbers n up to 127 of 2^(e - 6). The inner sum is min(n, 0) . least +
// max(n, 0) . largest: a matrix product of fp16 numbers whose partial sums are whole and
// below 2 * 128 * 127^2 < 2^23, so exact in the accumulators whatever their order; one
// rounding follows (times the page's scale). The scores are the same on every run and machine,
// and so are the pages that they choose. 16 pages to a warp and instruction, 8 rows beside them.
// ONE: at most 8 rows, which take a page's bounds as they come; more go over them tile by tile
// from registers. 16 sequences of 35,000 to 60,001 tokens in pages of 32, 8 heads of 128, 4 rows a
// head (49 MB of bounds): 16 us, 3.1 TB/s, in L2 or not; bound by the look-ups before a block's
// first bounds and by five blocks an SM that each wait for theirs.
template <int D, int DT, bool ONE>
__global__ void __launch_bounds__(SCORE_THREADS, ONE ? 5 : 4) kv_score_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int K = 2 * D, STEPS = K / 16;
  __shared__ int64_t prefix[SLAB_BATCH + 1];
  constexpr int HELD = ONE ? 8 : ROWS;
  __shared__ uint2 rows[HELD / 8][STEPS][32];  // the second operand as the lanes hold it
  __shared__ float unit[HELD];                 // 2^(e - 6); NaN: no such row
  const ibp_kv_cache &c = a.c;
  const int P = c.page_tokens, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int group = a.q.q_heads / c.n_heads;
  grid_dependency_wait();  // for the kernel before it, most often that of the bounds
  grid_launch_dependents();
  auto chunks_of = [&](int b, int32_t *status) {
    int64_t row0;
    const int n = rows_at(a, b, &row0, status), pages = (kv_len(c, b, status) + P - 1) / P;
    return n > 0 && pages > a.pages ? (pages + CHUNK - 1) / CHUNK : 0;  // all are taken otherwise
  };
  if (threadIdx.x < 32)
    count_items(prefix, a.batch, [&](int b) {
      return (int64_t)chunks_of(a.b0 + b, blockIdx.x == 0 ? a.status : nullptr) * c.n_heads;
    });
  __syncthreads();
  const int64_t total = prefix[a.batch];
  const int64_t begin = total * blockIdx.x / gridDim.x, end = total * (blockIdx.x + 1) / gridDim.x;
  int ready_b = -1, ready_head = -1;
  struct Item {
    int b, head, col, n, pages;  // col: of this lane's first page
    int64_t row0;
    int page[2];  // of columns col and col + 8
  };
  auto look_up = [&](int64_t x) {
    Item t = {-1, 0, 0, 0, 0, 0, {-1, -1}};
    if (x >= end) return t;
    const int at = find_sequence(prefix, a.batch, x);
    const uint32_t chunks = (uint32_t)(prefix[at + 1] - prefix[at]) / (uint32_t)c.n_heads;
    const uint32_t in = (uint32_t)(x - prefix[at]);  // (one float of scratch a page, so far below 2^32)
    t.b = a.b0 + at;
    t.head = (int)(in / chunks);
    t.col = (int)(in % chunks) * CHUNK + warp * 16 + g;
    t.n = rows_at(a, t.b, &t.row0, nullptr);
    t.pages = (kv_len(c, t.b, nullptr) + P - 1) / P;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (t.col + 8 * h < t.pages) t.page[h] = kv_page(c, t.b, t.col + 8 * h, t4 == 0 ? a.status : nullptr);
    return t;
  };
  Item next = look_up(begin);  // the next item's pages are looked up before this one's scores
  for (int64_t x = begin; x < end; ++x) {
    const Item t = next;
    const int b = t.b, head = t.head, all = t.n * group, col = t.col, pages = t.pages;
    const int64_t row0 = t.row0;
    Pages16<D> p;
    p.load(a, t.page, head);
    next = look_up(x + 1);
    uint32_t m[ONE ? 1 : STEPS][4];
    if constexpr (!ONE)
#pragma unroll
      for (int k = 0; k < STEPS; ++k) p.operand(k, m[k]);
    float best[2] = {-INFINITY, -INFINITY};
    for (int r0 = 0; r0 < all; r0 += HELD) {
      const int some = min(all - r0, HELD), tiles = (some + 7) / 8;
      if (ready_b != b || ready_head != head || all > HELD) {
        __syncthreads();  // the ones before have been read
        rows_in_whole_numbers<D, DT, ONE, SCORE_WARPS>(a, row0, head, r0, some, tiles, rows, unit);
        __syncthreads();
        ready_b = b;
        ready_head = head;
      }
      p.template against<ONE>(best, m, tiles, rows, unit);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float score = p.score(best[h], h);
      if (t4 == 0 && col + 8 * h < pages)
        a.scores[((int64_t)b * c.n_heads + head) * c.table_cols + col + 8 * h] = score;
    }
  }
}

// ---- the highest scores ------------------------------------------------------------

constexpr int PICK_THREADS = 256, PICK_WARPS = PICK_THREADS / 32;
constexpr int BIN_BITS = 8, BINS = 1 << BIN_BITS;
constexpr int KEPT_KEYS = 8192;  // keys held in shared memory; of longer lists they are read again

// Unsigned order of the scores: NaN lowest, -0 = 0.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The columns of one (sequence, head) in rising order: the first, those of the rows' own pages,
// and of the others the `need` of the highest scores, lowest column first among equals: the
// need-th largest key is found from the top bits of the keys' own range down, 8 at a time (of
// floats of similar sizes the uppermost bits are the same: counting by those would queue at a
// few counters), then the keys above it and the first of those equal to it are listed in order.
struct Picking {
  uint32_t hist[BINS], warp_sum[PICK_WARPS], found[2];
  uint2 warp_count[PICK_WARPS];
};
// key_at(i): of column 1 + i, there for all threads of the block.
template <typename Keys>
__device__ __forceinline__ void pick_columns(int32_t *out, int open, int room, Picking &sm, Keys key_at) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // A key to a thread while there are few: its rank is counted (62 keys 4.5 us, 5.4 by their bits;
  // 217 keys 6.7 and 5.7).
  if (open <= 128) {
    const uint32_t mine = tid < open ? key_at(tid) : 0u;
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < open; ++i) {
      const uint32_t other = key_at(i);
      rank += other > mine || (other == mine && i < tid);
    }
    const bool chosen = tid < open && rank < room;
    const unsigned votes = __ballot_sync(FULL, chosen);
    if (lane == 0) sm.warp_sum[warp] = __popc(votes);
    __syncthreads();
    int to = 1 + __popc(votes & ((1u << lane) - 1u));
    for (int k = 0; k < warp; ++k) to += sm.warp_sum[k];
    if (chosen) out[to] = 1 + tid;
    return;
  }
  // the keys' range
  uint32_t least = FULL, most = 0;
  for (int i = tid; i < open; i += PICK_THREADS) {
    const uint32_t key = key_at(i);
    least = min(least, key);
    most = max(most, key);
  }
  least = __reduce_min_sync(FULL, least);
  most = __reduce_max_sync(FULL, most);
  if (lane == 0) sm.warp_count[warp] = make_uint2(least, most);
  __syncthreads();
  for (int k = 0; k < PICK_WARPS; ++k) {
    least = min(least, sm.warp_count[k].x);
    most = max(most, sm.warp_count[k].y);
  }
  __syncthreads();  // (its places are used again)
  uint32_t need = (uint32_t)room, value = 0;  // of key - least, from its top bits down
  for (int top = 32 - __clz((int)(most - least)), shift; room > 0 && top > 0; top = shift) {
    shift = max(top - BIN_BITS, 0);
    for (int i = tid; i < BINS; i += PICK_THREADS) sm.hist[i] = 0;
    __syncthreads();
    const uint32_t above = top >= 32 ? 0u : value >> top;
    for (int i = tid; i < open; i += PICK_THREADS) {
      const uint32_t d = key_at(i) - least;
      if ((top >= 32 ? 0u : d >> top) == above) atomicAdd(&sm.hist[(d >> shift) & (BINS - 1)], 1u);
    }
    __syncthreads();
    // bins from the top, a few to a thread
    constexpr int EACH = BINS / PICK_THREADS;
    uint32_t mine[EACH], sum = 0;
#pragma unroll
    for (int e = 0; e < EACH; ++e) sum += mine[e] = sm.hist[BINS - 1 - (EACH * tid + e)];
    uint32_t run = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(FULL, run, o);
      if (lane >= o) run += y;
    }
    if (lane == 31) sm.warp_sum[warp] = run;
    __syncthreads();
    uint32_t before = run - sum;
    for (int k = 0; k < warp; ++k) before += sm.warp_sum[k];
#pragma unroll
    for (int e = 0; e < EACH; ++e) {
      if (before < need && before + mine[e] >= need) {
        sm.found[0] = (uint32_t)(BINS - 1 - (EACH * tid + e));
        sm.found[1] = need - before;
      }
      before += mine[e];
    }
    __syncthreads();
    value = (shift + BIN_BITS >= 32 ? 0u : value >> (shift + BIN_BITS) << (shift + BIN_BITS)) | sm.found[0] << shift;
    need = sm.found[1];
  }
  const uint32_t prefix = least + value;
  // each warp a stretch of columns: what lies above the threshold and at it
  const int per_warp = (open + 32 * PICK_WARPS - 1) / (32 * PICK_WARPS) * 32;
  const int first = min(warp * per_warp, open), last = min(first + per_warp, open);
  uint32_t gt = 0, eq = 0;
  for (int t0 = first; t0 < last; t0 += 32) {
    const uint32_t key = t0 + lane < last ? key_at(t0 + lane) : 0u;
    gt += __popc(__ballot_sync(FULL, t0 + lane < last && key > prefix));
    eq += __popc(__ballot_sync(FULL, t0 + lane < last && key == prefix));
  }
  if (lane == 0) sm.warp_count[warp] = make_uint2(gt, eq);
  __syncthreads();
  uint32_t gt_before = 0, eq_before = 0;
  for (int k = 0; k < warp; ++k) {
    gt_before += sm.warp_count[k].x;
    eq_before += sm.warp_count[k].y;
  }
  if (room == 0) return;
  const uint32_t lower = (1u << lane) - 1u;
  for (int t0 = first; t0 < last; t0 += 32) {
    const bool in = t0 + lane < last;
    const uint32_t key = in ? key_at(t0 + lane) : 0u;
    const unsigned above_it = __ballot_sync(FULL, in && key > prefix), at_it = __ballot_sync(FULL, in && key == prefix);
    const uint32_t g = gt_before + __popc(above_it & lower), e = eq_before + __popc(at_it & lower);
    if (in && (key > prefix || (key == prefix && e < need))) {
      const uint32_t to = g + min(e, need);
      if (to < (uint32_t)room) out[1 + to] = 1 + t0 + lane;
    }
    gt_before += __popc(above_it);
    eq_before += __popc(at_it);
  }
}

// What needs no score: all columns of a list that holds them, the first and the rows' own of
// another. Whether others compete.
__device__ __forceinline__ bool sure_columns(int32_t *out, const PageList &p, int pages) {
  const int tid = threadIdx.x;
  for (int i = p.count + tid; i < pages; i += PICK_THREADS) out[i] = -1;
  if (p.count == p.all) {
    for (int i = tid; i < p.all; i += PICK_THREADS) out[i] = i;
    return false;
  }
  // p.all > pages >= first + own: columns 1 .. first_own - 1 compete
  const int own = p.all - p.first_own;
  if (tid == 0) out[0] = 0;
  for (int i = tid; i < own; i += PICK_THREADS) out[pages - own + i] = p.first_own + i;
  return true;
}

__global__ void __launch_bounds__(PICK_THREADS) kv_pick_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ uint32_t keys[KEPT_KEYS];
  __shared__ Picking sm;
  const ibp_kv_cache &c = a.c;
  const int b = a.b0 + blockIdx.x / c.n_heads, head = blockIdx.x % c.n_heads, tid = threadIdx.x;
  const int64_t list = (int64_t)b * c.n_heads + head;
  int32_t *out = a.columns + list * a.pages;
  int64_t row0;
  const int n = rows_at(a, b, &row0, nullptr), len = n > 0 ? kv_len(c, b, nullptr) : 0;
  const PageList p = page_list(c, len, n, a.pages);
  grid_dependency_wait();
  grid_launch_dependents();
  if (!sure_columns(out, p, a.pages)) return;
  const int room = a.pages - (p.all - p.first_own) - 1, open = p.first_own - 1;
  const float *scores = a.scores + list * c.table_cols + 1;
  const bool held = open <= KEPT_KEYS;
  if (held)
    for (int i = tid; i < open; i += PICK_THREADS) keys[i] = score_key(__ldcg(scores + i));
  __syncthreads();
  pick_columns(out, open, room, sm, [&](int i) { return held ? keys[i] : score_key(__ldcg(scores + i)); });
}

// Both for lists of few pages, a block to a (sequence, head): one launch, and no score leaves the
// SM. Few long lists need more blocks than there are lists.
constexpr int SHORT_LIST = 1024;
template <int D, int DT, bool ONE>
__global__ void __launch_bounds__(PICK_THREADS, 2) kv_select_short_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int STEPS = D / 8, HELD = ONE ? 8 : ROWS;
  __shared__ uint2 rows[HELD / 8][STEPS][32];
  __shared__ float unit[HELD];
  __shared__ uint32_t keys[SHORT_LIST];
  __shared__ Picking sm;
  const ibp_kv_cache &c = a.c;
  const int b = a.b0 + blockIdx.x / c.n_heads, head = blockIdx.x % c.n_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  int32_t *status = head == 0 && threadIdx.x == 0 ? a.status : nullptr;
  grid_dependency_wait();  // for the kernel before it, most often that of the bounds
  grid_launch_dependents();
  int32_t *out = a.columns + ((int64_t)b * c.n_heads + head) * a.pages;
  int64_t row0;
  const int n = rows_at(a, b, &row0, status), held = kv_len(c, b, status), all = n * (a.q.q_heads / c.n_heads);
  const PageList p = page_list(c, n > 0 ? held : 0, n, a.pages);
  if (!sure_columns(out, p, a.pages)) return;
  const int room = a.pages - (p.all - p.first_own) - 1, open = p.first_own - 1;
  const int passes = (p.all + 16 * PICK_WARPS - 1) / (16 * PICK_WARPS);
  // page ids are looked up two passes ahead of their scores, bounds one
  auto look_up = [&](int pass, int *page) {
    const int col = (pass * PICK_WARPS + warp) * 16 + g;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      page[h] = col + 8 * h < p.all ? kv_page(c, b, col + 8 * h, t4 == 0 ? a.status : nullptr) : -1;
  };
  Pages16<D> q, next;
  int page[2];
  look_up(0, page);
  next.load(a, page, head);
  look_up(1, page);
  for (int pass = 0; pass < passes; ++pass) {
    const int col = (pass * PICK_WARPS + warp) * 16 + g;
    q = next;
    if constexpr (ONE) {  // (more rows need the registers)
      next.load(a, page, head);
      look_up(pass + 2, page);
    }
    uint32_t m[ONE ? 1 : STEPS][4];
    if constexpr (!ONE)
#pragma unroll
      for (int k = 0; k < STEPS; ++k) q.operand(k, m[k]);
    float best[2] = {-INFINITY, -INFINITY};
    for (int r0 = 0; r0 < all; r0 += HELD) {
      const int some = min(all - r0, HELD), tiles = (some + 7) / 8;
      if (pass == 0 || all > HELD) {
        __syncthreads();  // the ones before have been read
        rows_in_whole_numbers<D, DT, ONE, PICK_WARPS>(a, row0, head, r0, some, tiles, rows, unit);
        __syncthreads();
      }
      q.template against<ONE>(best, m, tiles, rows, unit);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float score = q.score(best[h], h);
      const int at = col + 8 * h - 1;
      if (t4 == 0 && at >= 0 && at < open) keys[at] = score_key(score);
    }
    if constexpr (!ONE) {
      next.load(a, page, head);
      look_up(pass + 2, page);
    }
  }
  __syncthreads();
  pick_columns(out, open, room, sm, [&](int i) { return keys[i]; });
}

template <int D>
int launch_bounds_of(BoundsArgs a, const DeviceInfo &dev, cudaStream_t s) {
  const auto kernel = a.c.code == IBP_KV_INT8 ? kv_bounds_kernel<D, IBP_KV_INT8> : kv_bounds_kernel<D, IBP_KV_E4M3>;
  for (a.b0 = 0; a.b0 < a.c.batch; a.b0 += SLAB_BATCH) {
    a.batch = std::min(a.c.batch - a.b0, SLAB_BATCH);
    const int64_t most = ((int64_t)a.batch * a.c.n_heads * a.c.table_cols + BOUNDS_THREADS / 32 - 1) / (BOUNDS_THREADS / 32);
    const int64_t ctas = std::min<int64_t>(most, dev.sm_count * 3);
    kernel<<<(unsigned)ctas, BOUNDS_THREADS, 0, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return IBP_ERR_CUDA;
  }
  return IBP_OK;
}

}  // namespace

int launch_kv_bounds(const ibp_kv_cache &c, int8_t *d_bounds, const int32_t *d_begin, int32_t *d_status,
                     cudaStream_t s) {
  if (c.table_cols == 0) return IBP_OK;
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  BoundsArgs a = {c, d_bounds, d_begin, d_status, 0, 0};
  return c.head_dim == 64 ? launch_bounds_of<64>(a, dev, s) : launch_bounds_of<128>(a, dev, s);
}

size_t kv_select_scratch_bytes(const ibp_kv_cache &c) {
  return ((size_t)c.batch * c.n_heads * c.table_cols * sizeof(float) + 15) / 16 * 16;
}

int launch_kv_select(const ibp_kv_cache &c, const int8_t *d_bounds, const ibp_kv_query &query, int64_t pages,
                     int32_t *d_columns, void *d_scratch, int32_t *d_status, cudaStream_t s) {
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  SelectArgs a = {};
  a.c = c;
  a.q = query;
  a.q.max_q = std::min(query.max_q, query.n_rows);
  a.bounds = d_bounds;
  a.scores = static_cast<float *>(d_scratch);
  a.columns = d_columns;
  a.status = d_status;
  a.pages = (int)pages;
  for (a.b0 = 0; a.b0 < c.batch; a.b0 += SLAB_BATCH) {
    a.batch = std::min(c.batch - a.b0, SLAB_BATCH);
    const bool one = a.q.max_q * (query.q_heads / c.n_heads) <= 8, bf16 = query.dtype == IBP_BF16;
    // One kernel where a block is done with its list in two passes of 128 pages, or where there are
    // lists for all SMs (whole steps in one | two kernels: 256 lists of 64 pages 57 | 62 us, 192 of up
    // to 219 42 | 48, 8 of 487 26.6 | 24.6).
    const bool lists = (int64_t)a.batch * c.n_heads >= dev.sm_count;
    if (c.table_cols <= 2 * 16 * PICK_WARPS || (lists && c.table_cols <= SHORT_LIST)) {
      const auto kernel =
          c.head_dim == 64
              ? (one ? (bf16 ? kv_select_short_kernel<64, IBP_BF16, true> : kv_select_short_kernel<64, IBP_FP16, true>)
                     : (bf16 ? kv_select_short_kernel<64, IBP_BF16, false> : kv_select_short_kernel<64, IBP_FP16, false>))
              : (one ? (bf16 ? kv_select_short_kernel<128, IBP_BF16, true> : kv_select_short_kernel<128, IBP_FP16, true>)
                     : (bf16 ? kv_select_short_kernel<128, IBP_BF16, false> : kv_select_short_kernel<128, IBP_FP16, false>));
      if (launch_dependent(kernel, dim3((unsigned)(a.batch * c.n_heads)), dim3(PICK_THREADS), 0, s, a) != cudaSuccess)
        return IBP_ERR_CUDA;
      continue;
    }
    const int64_t most = (int64_t)a.batch * c.n_heads * ((c.table_cols + CHUNK - 1) / CHUNK);
    const auto kernel =
        c.head_dim == 64
            ? (one ? (bf16 ? kv_score_kernel<64, IBP_BF16, true> : kv_score_kernel<64, IBP_FP16, true>)
                   : (bf16 ? kv_score_kernel<64, IBP_BF16, false> : kv_score_kernel<64, IBP_FP16, false>))
            : (one ? (bf16 ? kv_score_kernel<128, IBP_BF16, true> : kv_score_kernel<128, IBP_FP16, true>)
                   : (bf16 ? kv_score_kernel<128, IBP_BF16, false> : kv_score_kernel<128, IBP_FP16, false>));
    const int64_t ctas = std::max<int64_t>(std::min<int64_t>(most, dev.sm_count * (one ? 5 : 4)), 1);
    if (launch_dependent(kernel, dim3((unsigned)ctas), dim3(SCORE_THREADS), 0, s, a) != cudaSuccess) return IBP_ERR_CUDA;
    if (launch_dependent(kv_pick_kernel, dim3((unsigned)(a.batch * c.n_heads)), dim3(PICK_THREADS), 0, s, a) !=
        cudaSuccess)
      return IBP_ERR_CUDA;
  }
  return IBP_OK;
}

}  // namespace ibp
