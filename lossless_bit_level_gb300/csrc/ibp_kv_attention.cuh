// Shared by the attention kernels of the 8-bit paged key/value cache: how a launch is
// divided over the GPU, and the kernel that joins what was divided.
#pragma once

#include "ibp_kv_device.cuh"

namespace ibp {

namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float NONE = -1e30f;  // reference of a row that has seen no token yet
// A reference of the second product is set so that the largest factor is 2^SHIFT: fp16
// then holds factors 2^-31 of the largest, and there is room for it to grow by 2^8.
constexpr float SHIFT = 7.0f;

constexpr int MAX_BATCH = 256;  // sequences of one launch (their tile counts are in shared memory)
constexpr int MAX_CTAS = 512;          // three to each of 152 SMs, and some
constexpr int MAX_PREFILL_CTAS = 160;  // one to an SM

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Before a CTA ends: waits for a barrier that copies or matrix instructions in flight complete
// by themselves. They do so within microseconds; the limit is its own, far above that of the
// waits that may have run out before, and what it leaves undone is recorded.
constexpr uint64_t DRAIN_NS = 5 * WAIT_TIMEOUT_NS;
__device__ __forceinline__ void drain(uint64_t *bar, uint32_t parity, int32_t *status) {
  if (!mbar_wait(bar, parity, nullptr, DRAIN_NS)) report(status, IBP_ERR_TIMEOUT);
}

// Orders this thread's shared-memory accesses before later bulk copies into the same place.
__device__ __forceinline__ void fence_async_proxy() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// What the joining kernel for many rows needs of a CTA's place: the segment its stretch
// begins in (tile: how many of the segment's tiles lie before it; 0: none).
struct Cut {
  int64_t total;  // tiles of the launch
  int b, head, block, tile, tiles, unused;
};

struct AttentionArgs {
  ibp_kv_cache c;
  ibp_kv_query q;
  int32_t *status;
  uint64_t wait_ns;
  int withhold;     // testing: fetch the first tile of a stretch only
  int b0, batch, ctas, score_cols;
  int slice0, slice_rows;  // rows of a sequence that this launch is for (slice_rows 0: all)
  float *part;      // [ctas][2] partial results: MB rows of D values, then MB of (m, mv, l, 0)
  float *lse2;      // of segments that one CTA finished, in the order of score_row
  float *scores;    // [rows * q_heads][score_cols] in that order, or null
  Cut *cuts;        // [ctas] (many rows)
};

struct Sequence {
  int64_t row0;  // its first query row
  int n, len;    // query rows, tokens
};

__device__ __forceinline__ Sequence sequence_of(const AttentionArgs &a, int b, int32_t *status) {
  Sequence s;
  int64_t lo, hi;
  kv_row_range(a.q.d_cu, a.q.n_rows, a.q.max_q, a.b0 + b, status, &lo, &hi);
  if (hi - lo > a.q.max_q) {
    report(status, IBP_ERR_INDEX);
    hi = lo + a.q.max_q;
  }
  s.row0 = lo;
  s.n = (int)(hi - lo);
  s.len = kv_len(a.c, a.b0 + b, status);
  return s;
}

// The rows of a sequence that the launch is for: all but where scores are kept for the weights
// and those of all rows would take too much room.
struct Slice : Sequence {
  int at;  // position of the first of them: row i sees the tokens up to at + i
};
template <bool SCORES>
__device__ __forceinline__ Slice slice_of(const AttentionArgs &a, int b, int32_t *status) {
  Slice s;
  static_cast<Sequence &>(s) = sequence_of(a, b, status);
  s.at = s.len - s.n;
  if (SCORES && a.slice_rows) {
    const int skip = min(a.slice0, s.n);
    s.row0 += skip;
    s.at += skip;
    s.n = min(s.n - skip, a.slice_rows);
  }
  return s;
}

// The rows of one K/V head of sequence b, row by row: where their scores begin.
__device__ __forceinline__ int64_t score_row(const AttentionArgs &a, const Slice &s, int b, int head) {
  const int64_t row = a.slice_rows ? (int64_t)b * a.slice_rows : s.row0;
  return row * a.q.q_heads + (int64_t)head * s.n * (a.q.q_heads / a.c.n_heads);
}

// How a launch is divided. A (sequence, K/V head, block of MB query rows) is a segment of
// tiles of TILE tokens; all tiles of all segments are laid end to end (sequence, head,
// block, token) and every CTA takes an equal stretch, so a batch of any mix of lengths
// fills the GPU and a segment is joined from as many CTAs as it took.
struct Split {
  int64_t total;
  int ctas;  // that have work: every one of them has a tile at least
  __device__ __forceinline__ Split(int64_t tiles, int launched)
      : total(tiles), ctas((int)min((int64_t)launched, tiles)) {}
  __device__ __forceinline__ int64_t start(int cta) const { return total * cta / ctas; }
  // the CTA whose stretch holds tile x
  __device__ __forceinline__ int owner(int64_t x) const {
    return (int)(((x + 1) * ctas - 1) / total);
  }
};

// Tiles of a sequence's blocks. EvenPlan: every block goes over all tokens (few query
// rows: the last ones, so at most a tile is spared by their order).
template <int MB_, int TILE_>
struct EvenPlan {
  static constexpr int MB = MB_, TILE = TILE_;
  int blocks, tiles_each;
  __device__ __forceinline__ EvenPlan(const Sequence &s, int group)
      : blocks((s.n * group + MB - 1) / MB), tiles_each((s.len + TILE - 1) / TILE) {}
  __device__ __forceinline__ int tiles(int) const { return tiles_each; }
  __device__ __forceinline__ int64_t before(int block) const { return (int64_t)block * tiles_each; }
  // the block that holds tile x of a head
  __device__ __forceinline__ int find(int64_t x) const { return (int)(x / tiles_each); }
};

// CausalPlan: a block stops at the last token its last row sees. Block j's last query is
// q_j = (MB (j + 1) - 1) / group (the sequence's last for the last block), so it has
// floor((MB j + (len - n + TILE) group + MB - 1) / (TILE group)) tiles; their sum over j
// is a sum of floors of an arithmetic progression. The steps are the published ones: whole
// parts out, then slope and modulus change places as in Euclid's algorithm (Graham, Knuth and
// Patashnik, Concrete Mathematics, 3.5, reciprocity of such sums).
template <int MB_, int TILE_>
struct CausalPlan {
  static constexpr int MB = MB_, TILE = TILE_;
  int blocks, group, n, len;
  __device__ __forceinline__ CausalPlan(const Sequence &s, int g)
      : blocks((s.n * g + MB - 1) / MB), group(g), n(s.n), len(s.len) {}
  __device__ __forceinline__ int tiles(int block) const {
    const int last = block == blocks - 1 ? n - 1 : (MB * (block + 1) - 1) / group;
    return (max(len - n + last + 1, 0) + TILE - 1) / TILE;
  }
  __device__ __forceinline__ int64_t before(int block) const {
    // blocks whose last query sees nothing have no tiles
    const int64_t hidden = max((int64_t)(n - len) * group, (int64_t)0) / MB;
    const bool all = block == blocks;
    int64_t count = (all ? block - 1 : block) - hidden, sum = 0;
    if (count > 0) {
      int64_t m = (int64_t)TILE * group, a = MB;
      int64_t b = MB * hidden + (int64_t)(len - n + TILE) * group + MB - 1, k = count;
      for (;;) {
        sum += (k - 1) * k / 2 * (a / m) + k * (b / m);
        a %= m;
        b %= m;
        const int64_t y = a * k + b;
        if (y < m) break;
        k = y / m;
        b = y % m;
        const int64_t t = m;
        m = a;
        a = t;
      }
    }
    return all && blocks > 0 ? sum + tiles(blocks - 1) : sum;
  }
  __device__ __forceinline__ int find(int64_t x) const {
    int lo = 0, hi = blocks;  // the last block with before(block) <= x
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before(mid) <= x) lo = mid; else hi = mid;
    }
    return lo;
  }
};

__device__ __forceinline__ int find_sequence(const int64_t *prefix, int batch, int64_t x) {
  int lo = 0, hi = batch;  // the last b with prefix[b] <= x (empty ones come before it)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (prefix[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Where the parts of a segment lie. Only a segment's first CTA can have held another
// segment before it.
struct Parts {
  int first, last;  // CTAs
  int second;       // the first one's part is its second
};
__device__ __forceinline__ Parts parts_of(int64_t total, int64_t start, int tiles, int ctas) {
  const Split split(total, ctas);
  Parts p;
  p.first = split.owner(start);
  p.last = split.owner(start + tiles - 1);
  p.second = split.start(p.first) < start;
  return p;
}
template <int MB, int D>
__device__ __forceinline__ const float *part_at(const AttentionArgs &a, const Parts &p, int cta) {
  return a.part + ((int64_t)cta * 2 + (cta == p.first ? p.second : 0)) * ((int64_t)MB * (D + 4));
}

// (m, mv, l) of one row over all parts: a warp's lanes take every 32nd part, then a
// fixed tree.
template <int MB, int D>
__device__ __forceinline__ float4 join_row(const AttentionArgs &a, const Parts &p, int r) {
  float4 y = make_float4(NONE, NONE, 0.0f, 0.0f);
  for (int k = p.first + (int)(threadIdx.x & 31); k <= p.last; k += 32) {
    const float4 z = reinterpret_cast<const float4 *>(part_at<MB, D>(a, p, k) + MB * D)[r];
    const float m = fmaxf(y.x, z.x);
    y.z = y.z * exp2_fast(y.x - m) + z.z * exp2_fast(z.x - m);
    y.x = m;
    y.y = fmaxf(y.y, z.y);
  }
  for (int o = 16; o > 0; o >>= 1) {
    const float zx = __shfl_xor_sync(FULL, y.x, o), zl = __shfl_xor_sync(FULL, y.z, o);
    const float m = fmaxf(y.x, zx);
    y.y = fmaxf(y.y, __shfl_xor_sync(FULL, y.y, o));
    y.z = y.z * exp2_fast(y.x - m) + zl * exp2_fast(zx - m);
    y.x = m;
  }
  return y;
}

constexpr int FINISH_THREADS = 128;
constexpr int WEIGHT_CHUNKS = 2;  // of 4 tokens a thread
constexpr int WEIGHT_TOKENS = 4 * FINISH_THREADS * WEIGHT_CHUNKS;
// Parts loaded at a time: a long sequence with few rows is cut into dozens and waits for
// them in turn (120,001 and 70,000 tokens: 77 us with 4 at a time, 73 with 16). The CTAs
// that add up weights need the registers.
template <typename Plan, bool SCORES>
constexpr int JOIN_AHEAD = SCORES || Plan::MB > 16 ? 4 : 16;

// After few rows. Blocks x < row_blocks join the parts of one segment (and clear the rows
// of empty sequences): o = sum_k o_k 2^(mv_k - mv), l = sum_k l_k 2^(m_k - m) in the order of
// the parts, so that results do not depend on timing. The others add up the weights of
// WEIGHT_TOKENS tokens from the scores, p_t = 2^(score - log2 of the row's sum), rows in
// their order: once the sums are known, without atomics, and for what no row sees the
// score -inf gives 0. 48 ragged sequences of 28 rows, 4 heads (43 MB of scores, in L2 or
// HBM): 23 us alone, waiting for loads; it starts while the attending kernel ends. Every
// block waits for that kernel before it returns, with work or without: what comes next in
// the stream or a graph may be ordered behind this grid alone.
template <int D, int DT, typename Plan, bool SCORES>
__global__ void __launch_bounds__(FINISH_THREADS, (JOIN_AHEAD<Plan, SCORES>) > 4 ? 2 : 8)
    kv_finish_kernel(const __grid_constant__ AttentionArgs a, int row_blocks) {
  constexpr int MB = Plan::MB;
  __shared__ float lse2[MB];
  __shared__ Parts where;
  __shared__ int64_t prefix[2];  // tiles before sequence b and in all
  const int b = blockIdx.z, head = blockIdx.y;
  const int group = a.q.q_heads / a.c.n_heads;
  // what follows from the lengths alone is worked out before the attending kernel ends
  // (whatever wrote the lengths ended before that one began)
  const Slice s = slice_of<SCORES>(a, b, nullptr);
  const Plan plan(s, group);
  const int all = s.n * group;
  if (threadIdx.x < 32) {
    int64_t before = 0, total = 0;
    for (int k = threadIdx.x; k < a.batch; k += 32) {
      const Slice other = slice_of<SCORES>(a, k, nullptr);
      const Plan theirs(other, group);
      const int64_t tiles = a.c.n_heads * theirs.before(theirs.blocks);
      total += tiles;
      if (k < b) before += tiles;
    }
    for (int o = 16; o > 0; o >>= 1) {
      before += __shfl_xor_sync(FULL, before, o);
      total += __shfl_xor_sync(FULL, total, o);
    }
    if (threadIdx.x == 0) {
      prefix[0] = before;
      prefix[1] = total;
    }
  }
  __syncthreads();
  if ((int)blockIdx.x < row_blocks) {
    const int block = blockIdx.x, r0 = block * MB, rows = min(MB, all - r0);
    const int tiles = rows > 0 ? plan.tiles(block) : 0;
    if (threadIdx.x == 0 && tiles > 0)
      where = parts_of(prefix[1], prefix[0] + head * plan.before(plan.blocks) + plan.before(block),
                       tiles, a.ctas);
    __syncthreads();
    const Parts p = where;
    grid_dependency_wait();
    if (rows <= 0 || (tiles > 0 && p.first == p.last)) return;
    for (int u = threadIdx.x; u < rows * (D / 4); u += FINISH_THREADS) {
      const int r = u / (D / 4), piece = u % (D / 4), rr = r0 + r;
      const int64_t row = s.row0 + rr / group;
      const int qh = head * group + rr % group;
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float sum = 0.0f, top = 0.0f;
      if (tiles > 0) {
        // parts in the order of their CTAs, AHEAD of them loaded at a time
        constexpr int AHEAD = JOIN_AHEAD<Plan, SCORES>;
        float topv = NONE;
        top = NONE;
        for (int k0 = p.first; k0 <= p.last; k0 += AHEAD) {
          float4 st[AHEAD], z[AHEAD];
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {
            const float *part = part_at<MB, D>(a, p, min(k0 + k, p.last));
            st[k] = reinterpret_cast<const float4 *>(part + MB * D)[r];
            z[k] = reinterpret_cast<const float4 *>(part)[r * (D / 4) + piece];
          }
          float m = top, mv = topv;
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {
            m = fmaxf(m, st[k].x);  // a part read twice does not raise it
            mv = fmaxf(mv, st[k].y);
          }
          const float fl = exp2_fast(top - m), fo = exp2_fast(topv - mv);
          sum *= fl;
          y = make_float4(y.x * fo, y.y * fo, y.z * fo, y.w * fo);
#pragma unroll
          for (int k = 0; k < AHEAD; ++k)
            if (k0 + k <= p.last) {
              const float f = exp2_fast(st[k].y - mv);
              sum += st[k].z * exp2_fast(st[k].x - m);
              y.x += z[k].x * f;
              y.y += z[k].y * f;
              y.z += z[k].z * f;
              y.w += z[k].w * f;
            }
          top = m;
          topv = mv;
        }
        const float f = sum > 0.0f ? exp2_fast(topv - top) / sum : 0.0f;
        y = make_float4(y.x * f, y.y * f, y.z * f, y.w * f);
      }
      *reinterpret_cast<uint2 *>(static_cast<char *>(a.q.out) +
                                 2 * (row * a.q.out_row_stride + qh * a.q.out_head_stride + 4 * piece)) =
          make_uint2(pack2<DT>(y.x, y.y), pack2<DT>(y.z, y.w));
      if (piece == 0 && a.q.d_lse)
        a.q.d_lse[row * a.q.q_heads + qh] = sum > 0.0f ? (top + log2f(sum)) * LN2 : -INFINITY;
    }
    return;
  }
  if constexpr (SCORES) {
    const int t0 = ((int)blockIdx.x - row_blocks) * WEIGHT_TOKENS + 4 * (int)threadIdx.x;
    constexpr int STEP = 4 * FINISH_THREADS;
    const int64_t row0 = score_row(a, s, b, head);
    const int64_t at = ((int64_t)(a.b0 + b) * a.c.n_heads + head) * a.q.weights_stride + t0;
    float sum[WEIGHT_CHUNKS][4];
#pragma unroll
    for (int k = 0; k < WEIGHT_CHUNKS; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        sum[k][e] = a.q.d_weights_in && t0 + k * STEP + e < s.len
                        ? a.q.decay * a.q.d_weights_in[at + k * STEP + e]
                        : 0.0f;
    grid_dependency_wait();
    if (t0 - 4 * (int)threadIdx.x >= s.len) return;
    for (int r0 = 0; r0 < all; r0 += MB) {
      const int rows = min(MB, all - r0);
      const int block = r0 / MB;
      __syncthreads();
      if (threadIdx.x == 0)
        where = parts_of(prefix[1], prefix[0] + head * plan.before(plan.blocks) + plan.before(block),
                         plan.tiles(block), a.ctas);
      __syncthreads();
      const Parts p = where;
      for (int r = threadIdx.x >> 5; r < rows; r += FINISH_THREADS / 32) {
        float z;
        if (p.first == p.last) {
          z = a.lse2[row0 + r0 + r];
        } else {
          const float4 st = join_row<MB, D>(a, p, r);
          z = st.z > 0.0f ? st.x + log2f(st.z) : -INFINITY;
        }
        lse2[r] = z == -INFINITY ? INFINITY : z;  // a row that saw nothing adds nothing
      }
      __syncthreads();
      const float *from = a.scores + (row0 + r0) * a.score_cols + t0;
#pragma unroll 4
      for (int r = 0; r < rows; ++r, from += a.score_cols) {
        const float z = lse2[r];
#pragma unroll
        for (int k = 0; k < WEIGHT_CHUNKS; ++k)
          if (t0 + k * STEP < s.len) {
            const float4 x = *reinterpret_cast<const float4 *>(from + k * STEP);
            sum[k][0] += exp2_fast(x.x - z);
            sum[k][1] += exp2_fast(x.y - z);
            sum[k][2] += exp2_fast(x.z - z);
            sum[k][3] += exp2_fast(x.w - z);
          }
      }
    }
#pragma unroll
    for (int k = 0; k < WEIGHT_CHUNKS; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t0 + k * STEP + e < s.len) a.q.d_weights[at + k * STEP + e] = sum[k][e];
  }
}

}  // namespace

}  // namespace ibp
