// Attention over the 8-bit paged key/value cache (declared in include/ibp.h).
//
// out = sum_t p_t v_t, p = softmax of scale * q . k_t over the tokens a row sees, in one
// pass over the keys: with x = scale * log2(e) * q . k_t, a running reference m and
//   l = sum 2^(x - m),  o = sum 2^(x + log2 s_v - mv) c_v   (c_v: codes, s_v: their scale)
// both are multiplied by 2^(old - new) whenever a reference rises, and the output is
// o 2^(mv - m) / l. The value scale enters the exponent, with a reference mv of its own,
// so that the second product's factors stay within fp16 whatever the scales of the
// pages are; a reference only rises once the largest score has grown by 2^8 (a vote a slab
// instead of a maximum across lanes; fp16 and fp32 have the room).
//
// Roundings to fewer than 32 bits: codes become fp16 exactly; bf16 queries become fp16
// scaled by a power of two (exact to 2^-16 of a row's largest element); the second product's
// factors are rounded to fp16 (2^-11 of each), where the sum l adds the unrounded ones.
// Scores, references, sums and outputs are fp32 until the output is stored.
#include <algorithm>
#include <numeric>

#include "ibp_kv_attention.cuh"

namespace ibp {

namespace {

constexpr int TILE = 64;      // tokens a stage holds
constexpr int SLAB = 16;      // tokens a warp takes at a time; never more than one page
constexpr int CONSUMERS = 4;  // warps that compute; one more fetches
constexpr int THREADS = 32 * (CONSUMERS + 1);

__device__ __forceinline__ void mma16816(float *c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit elements held one row to four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Within a rare branch: keeps it from being turned into selects that every pass goes through.
__device__ __forceinline__ void stay_a_branch() { asm volatile("" ::: "memory"); }

// Codes to fp16, exactly. int8: the byte of code + 128 below 0x64 is 1024 + 128 + code (the
// well-known magic-number conversion: Warren, Hacker's Delight, chapter on floating point).
template <int CODE>
__device__ __forceinline__ uint32_t code_bias(uint32_t w) {
  return CODE == IBP_KV_INT8 ? w ^ 0x80808080u : w;
}
// Bytes 0, 1 (HIGH = 0) or 2, 3 of a biased word as two fp16.
template <int CODE, int HIGH>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  if constexpr (CODE == IBP_KV_INT8) {
    const uint32_t u = __byte_perm(w, 0x64646464u, HIGH ? 0x4342 : 0x4140);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&u), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    uint32_t y;
    const uint16_t x = HIGH ? (uint16_t)(w >> 16) : (uint16_t)w;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(x));
    return y;
  }
}

__device__ __forceinline__ void consumer_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * CONSUMERS) : "memory");
}

template <int D, int NT, int WQ>
struct Shape {
  using Plan = EvenPlan<8 * NT * WQ, TILE>;
  static constexpr int MB = 8 * NT * WQ;  // query rows of a segment
  // NT = 1 runs three CTAs on an SM (12 computing warps), NT = 2 two for its registers (three
  // with 64 elements a head measured no faster: 64.2 us against 63.0)
  static constexpr int per_sm = NT == 1 ? 3 : 2;
  static constexpr int STAGES = NT == 1 ? 4 : 6;
  static constexpr int stage_bytes = 2 * TILE * D;
  static constexpr int slabs = TILE / SLAB;
  static constexpr size_t part_floats = (size_t)MB * (D + 4);
  static constexpr size_t smem = (size_t)STAGES * stage_bytes + STAGES * slabs * 16 +
                                 3 * CONSUMERS * 8 * 4 +
                                 (2 * STAGES) * 8 + (MAX_BATCH + 1) * 8 + 16;
};

// What a consumer needs to know of 16 tokens in a stage.
struct __align__(16) SlabInfo {
  float ks, lv;  // key scale, log2 of the value scale
  int n;         // tokens held (0: the page is not there)
  int unused;
};

// Few query rows a K/V head: the cache is read once, 2 bytes of codes an element pair for
// 4 operations a row, so HBM should bound it. All (sequence, head, block of rows) segments
// lie end to end as tiles of 64 tokens and every CTA takes an equal stretch of them, so a
// batch of one long sequence fills the GPU as a ragged one does; a segment that lies in one
// stretch is finished here, the others leave parts that kv_finish_kernel joins. A producer
// warp brings tiles with bulk copies, 4 or 6 ahead; a consumer warp takes 16 tokens (all
// rows), computes K q^T and V^T p^T with mma.sync (rows are the narrow side, 8 at a time:
// the matrix unit's own 64 or 128 rows would be empty), WQ of them sharing the rows. What it
// turns into fp16 is shared by all rows.
//
// Measured, the whole call: 8 sequences of 4,096 tokens, 32 heads of 128, weights: 60 us
// (4.6 TB/s; floor 41); 2 sequences of 120,001 and 70,000 tokens, 8 heads: 73 us (5.3 TB/s;
// floor 57). What bounds it: 12 computing warps an SM (registers) that wait in turn for
// shared memory, conversions and exponentials (alone 53 us at 2.0 instructions a cycle, HBM
// 66 %; the long ones 67 us, HBM 74 %). 32 tokens a warp at a time measured slower (81 ->
// 113 us: only two tiles in flight); copies asked for before the scales gained nothing.
template <int D, int CODE, int DT, int NT, int WQ, bool SCORES>
__global__ void __launch_bounds__(THREADS, (Shape<D, NT, WQ>::per_sm))
    kv_attend_kernel(const __grid_constant__ AttentionArgs a) {
  using S = Shape<D, NT, WQ>;
  using Plan = typename S::Plan;
  constexpr int MB = S::MB, ST = S::STAGES, NS = S::slabs, J = D / 64, MT = D / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char *stages = smem;
  SlabInfo *slabs = reinterpret_cast<SlabInfo *>(smem + ST * S::stage_bytes);
  float *st_m = reinterpret_cast<float *>(slabs + ST * NS), *st_mv = st_m + CONSUMERS * 8,
        *st_l = st_mv + CONSUMERS * 8;
  uint64_t *full = reinterpret_cast<uint64_t *>(st_l + CONSUMERS * 8), *freed = full + ST;
  int64_t *prefix = reinterpret_cast<int64_t *>(freed + ST);
  volatile int *abort = reinterpret_cast<volatile int *>(prefix + MAX_BATCH + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ibp_kv_cache &c = a.c;
  const int group = a.q.q_heads / c.n_heads, cta = blockIdx.x;
  grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&freed[i], CONSUMERS);
    }
    *abort = 0;
    mbar_init_fence();
  }
  if (warp == CONSUMERS) {  // tiles before each sequence
    int64_t base = 0;
    for (int k0 = 0; k0 < a.batch; k0 += 32) {
      const int b = k0 + lane;
      int64_t tiles = 0;
      if (b < a.batch) {
        const Slice s = slice_of<SCORES>(a, b, cta == 0 ? a.status : nullptr);
        const Plan plan(s, group);
        tiles = c.n_heads * plan.before(plan.blocks);
      }
      int64_t sum = tiles;
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(FULL, sum, o);
        if (lane >= o) sum += y;
      }
      if (b < a.batch) prefix[b] = base + sum - tiles;
      base += __shfl_sync(FULL, sum, 31);
    }
    if (lane == 0) prefix[a.batch] = base;
  }
  __syncthreads();
  const int64_t total = prefix[a.batch];
  const Split split(total, a.ctas);
  if (cta >= split.ctas) return;
  const int64_t lo = split.start(cta), hi = split.start(cta + 1);

  if (warp == CONSUMERS) {
    // ---- the fetching warp: a lane looks up one piece (the part of a page that lies
    // in one tile) of the next 32, one batch ahead of the copies
    const int PP = min(c.page_tokens, TILE), NP = TILE / PP;
    const char *kc = static_cast<const char *>(c.k_codes), *vc = static_cast<const char *>(c.v_codes);
    const int64_t pieces = (hi - lo) * NP;
    struct Piece {
      int64_t at;  // byte offset of its codes, or -1
      float ks, lv;
      int n;       // tokens of it that the sequence holds
    };
    auto look_up = [&](int64_t e) {
      Piece p = {-1, 0.0f, 0.0f, 0};
      if (e >= pieces) return p;
      const int64_t x = lo + e / NP;
      const int b = find_sequence(prefix, a.batch, x);
      const int len = kv_len(c, a.b0 + b, nullptr), nt = (len + TILE - 1) / TILE;
      const int64_t local = x - prefix[b], per_head = (prefix[b + 1] - prefix[b]) / c.n_heads;
      const int head = (int)(local / per_head), tile = (int)(local % nt);
      const int t = tile * TILE + (int)(e % NP) * PP;
      if (t >= len) return p;
      const int page = kv_page(c, a.b0 + b, t / c.page_tokens, a.status);
      if (page < 0) return p;
      const int64_t si = (int64_t)page * c.n_heads + head;
      p.at = kv_tile(c, page, head) + (int64_t)(t % c.page_tokens) * D;
      p.ks = __ldg(c.k_scales + si);
      p.lv = log2f(__ldg(c.v_scales + si));
      p.n = min(len - t, PP);
      return p;
    };
    Piece next = look_up(lane), now = next;
    bool ok = true;
    int64_t i = 0;
    const int64_t upto = a.withhold ? 1 : hi - lo;
    for (; i < upto && ok; ++i) {
      const int s = (int)(i % ST), e = (int)((i * NP) & 31);
      if (e == 0) {
        now = next;
        next = look_up(i * NP + 32 + lane);
      }
      // (a warp whose wait ran out goes on freeing stages without having seen their tiles: after
      // that nothing is fetched into them, as its copies may be in flight still)
      if (i >= ST) ok = mbar_wait(&freed[s], (uint32_t)((i / ST) & 1) ^ 1u, abort, a.wait_ns) && !*abort;
      ok = __all_sync(FULL, ok);
      if (!ok) break;
      const int64_t at = __shfl_sync(FULL, now.at, e + lane % NP);
      const float ks = __shfl_sync(FULL, now.ks, e + lane % NP);
      const float lv = __shfl_sync(FULL, now.lv, e + lane % NP);
      const int n = __shfl_sync(FULL, now.n, e + lane % NP);
      const unsigned some = __ballot_sync(FULL, lane < NP && at >= 0);
      if (lane < NP) {
        for (int k = 0; k < PP / SLAB; ++k) {
          const SlabInfo info = {ks, lv, min(max(n - k * SLAB, 0), SLAB), 0};
          slabs[s * NS + lane * (PP / SLAB) + k] = info;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)(__popc(some) * 2 * PP * D));
      __syncwarp();
      if (lane < NP && at >= 0) {
        unsigned char *to = stages + s * S::stage_bytes + lane * PP * D;
        bulk_load(to, kc + at, PP * D, &full[s]);
        bulk_load(to + TILE * D, vc + at, PP * D, &full[s]);
      }
    }
    if (!ok && lane == 0) {
      report(a.status, IBP_ERR_TIMEOUT);
      *abort = 1;
    }
    // no copy may land after this CTA is gone, and the others may have stopped waiting for them
#pragma unroll 1
    for (int64_t k = i > ST ? i - ST : 0; k < i; ++k)
      drain(&full[k % ST], (uint32_t)((k / ST) & 1), a.status);
    return;
  }

  // ---- computing warps: S^T = K q^T (16 tokens x 8 NT rows), then O^T += V^T P^T
  const int g = lane >> 2, t4 = lane & 3;
  bool dead = false;  // a wait ran out: the rest is gone through without waiting or computing,
                      // so that no warp is missed at a barrier
  int64_t x = lo;
  int b = find_sequence(prefix, a.batch, lo), s = 0;
  uint32_t phase = 0;
  while (x < hi) {
    while (x >= prefix[b + 1]) ++b;
    const Slice sq = slice_of<SCORES>(a, b, nullptr);
    const Plan plan(sq, group);
    const int nt = plan.tiles_each, blocks = plan.blocks;
    const int64_t local = x - prefix[b];
    const int seg = (int)(local / nt), tile0 = (int)(local % nt);
    const int count = (int)min((int64_t)(nt - tile0), hi - x);
    const int head = seg / blocks, r0 = (seg % blocks) * MB, rows = min(MB, sq.n * group - r0);
    // as many warps side by side along the rows as these need, the others along a tile
    const int wqn = rows <= 8 * NT ? 1 : WQ >= 2 && rows <= 16 * NT ? 2 : WQ;
    const int wq = warp % wqn, wk = warp / wqn, wkn = CONSUMERS / wqn;
    const bool active = wq * 8 * NT < rows;

    // query rows as the second operand: lane (g, t) holds 16 consecutive elements of row g
    uint32_t qb[NT][MT][2];
    float rowc[NT][2];
    int limit[NT][2], least = 0x7FFFFFFF;
    // Where a lane's scores go: a K/V head's rows of a sequence lie one after another, so that
    // at 128 elements a head one address serves them all (one a row spills: 91 -> 74 us for 16
    // rows of 128 heads over 4,096 tokens; at 64 elements
    // one a row is faster: 85 -> 80 us for 48 ragged sequences).
    constexpr bool ONE = D == 128;
    float *score[ONE ? 1 : NT][ONE ? 1 : 2] = {};
    if constexpr (SCORES)
#pragma unroll
      for (int k = 0; k < (ONE ? 1 : NT); ++k)
#pragma unroll
        for (int w = 0; w < (ONE ? 1 : 2); ++w)
          score[k][w] = a.scores +
                        (score_row(a, sq, b, head) + r0 + wq * 8 * NT + 8 * k + 2 * t4 + w) * a.score_cols + g;
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      const int r = wq * 8 * NT + 8 * k + g;
      const bool live = r < rows;
      const int rr = r0 + r;
      const char *src = static_cast<const char *>(a.q.q) +
                        2 * ((sq.row0 + rr / group) * a.q.q_row_stride +
                             (head * group + rr % group) * a.q.q_head_stride);
      float big = 0.0f, y[J][16];
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[j][e] = 0.0f;
        if (live) load16<DT>(src + 2 * 16 * (t4 + 4 * j), y[j]);
#pragma unroll
        for (int e = 0; e < 16; ++e) big = fmaxf(big, fabsf(y[j][e]));
      }
      float up = 1.0f, down = 1.0f;
      if constexpr (DT == IBP_BF16) {
        // bf16 rows in fp16: brought to a largest magnitude in [1, 2) by a power of two,
        // which the score's factor takes back; elements 2^-16 of it and up stay exact
        big = fmaxf(big, __shfl_xor_sync(FULL, big, 1));
        big = fmaxf(big, __shfl_xor_sync(FULL, big, 2));
        const int e = min(max((int)(__float_as_uint(big) >> 23) - 127, -120), 120);
        up = __uint_as_float((uint32_t)(127 - e) << 23);
        down = __uint_as_float((uint32_t)(127 + e) << 23);
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          qb[k][4 * j + e][0] = pack2<IBP_FP16>(y[j][4 * e] * up, y[j][4 * e + 1] * up);
          qb[k][4 * j + e][1] = pack2<IBP_FP16>(y[j][4 * e + 2] * up, y[j][4 * e + 3] * up);
        }
      const float factor = down * (a.q.scale * LOG2E);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int col = wq * 8 * NT + 8 * k + 2 * t4 + w, cc = r0 + col;
        rowc[k][w] = __shfl_sync(FULL, factor, (2 * t4 + w) * 4);
        limit[k][w] = col < rows ? max(sq.at + cc / group + 1, 0) : 0x7FFFFFFF;
        least = min(least, limit[k][w]);
      }
    }
    for (int o = 1; o < 4; o <<= 1) least = min(least, __shfl_xor_sync(FULL, least, o));

    float o[NT][MT][4], m[NT][2], mv[NT][2], l[NT][2];
#pragma unroll
    for (int k = 0; k < NT; ++k) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        m[k][w] = mv[k][w] = NONE;
        l[k][w] = 0.0f;
      }
#pragma unroll
      for (int n = 0; n < MT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[k][n][e] = 0.0f;
    }

    for (int tile = tile0;; ++tile) {
      if (!dead && !__all_sync(FULL, mbar_wait(&full[s], phase, abort, a.wait_ns))) {
        dead = true;
        if (lane == 0) {
          report(a.status, IBP_ERR_TIMEOUT);
          *abort = 1;
        }
      }
      const unsigned char *kt = stages + s * S::stage_bytes, *vt = kt + TILE * D;
      for (int slab = wk; active && !dead && slab < NS; slab += wkn) {
        const int t0 = tile * TILE + slab * SLAB;
        if (t0 >= sq.len) break;
        const SlabInfo info = slabs[s * NS + slab];
        const bool whole = info.n == SLAB && t0 + SLAB <= least;
        // values: lane (g, t) holds D/8 consecutive elements of tokens 2t, 2t+1, 2t+8, 2t+9;
        // asked for before the scores where registers allow (82 -> 78 us for 48 ragged
        // sequences of 64 elements a head; at 128 they spill: 61 -> 65 us for a layer)
        constexpr bool EARLY = D == 64;
        uint32_t v[4][D / 32];
        auto load_values = [&] {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = 2 * t4 + (e & 1) + 8 * (e >> 1);
            const unsigned char *p = vt + (slab * SLAB + row) * D + g * (D / 8);
            if constexpr (D == 128) {
              const uint4 w = *reinterpret_cast<const uint4 *>(p);
              v[e][0] = w.x; v[e][1] = w.y; v[e][2] = w.z; v[e][3] = w.w;
            } else {
              const uint2 w = *reinterpret_cast<const uint2 *>(p);
              v[e][0] = w.x; v[e][1] = w.y;
            }
          }
          if (!whole) {  // what lies past the length is not a number of ours
            stay_a_branch();
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (2 * t4 + (e & 1) + 8 * (e >> 1) >= info.n)
#pragma unroll
                for (int w = 0; w < D / 32; ++w) v[e][w] = 0u;
          }
        };
        if constexpr (EARLY) load_values();
        // two chains of products, added at the end: a chain waits for each of its own
        float acc[NT][4], odd[NT][4];
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[k][e] = odd[k][e] = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const unsigned char *at = kt + (slab * SLAB + g) * D + 16 * (t4 + 4 * j);
          const uint4 ra = *reinterpret_cast<const uint4 *>(at);
          const uint4 rb = *reinterpret_cast<const uint4 *>(at + 8 * D);
          const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t ua = code_bias<CODE>(wa[e]), ub = code_bias<CODE>(wb[e]);
            const uint32_t a0 = code_pair<CODE, 0>(ua), a1 = code_pair<CODE, 0>(ub),
                           a2 = code_pair<CODE, 1>(ua), a3 = code_pair<CODE, 1>(ub);
#pragma unroll
            for (int k = 0; k < NT; ++k)
              mma16816(e & 1 ? odd[k] : acc[k], a0, a1, a2, a3, qb[k][4 * j + e][0], qb[k][4 * j + e][1]);
          }
        }
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[k][e] += odd[k][e];
        // scores of tokens g, g + 8 and rows 2t, 2t + 1
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const float f = rowc[k][w] * info.ks;
            acc[k][w] *= f;
            acc[k][w + 2] *= f;
          }
        if (!whole) {
          stay_a_branch();
#pragma unroll
          for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const int seen = min(limit[k][w] - t0, info.n);
              if (g >= seen) acc[k][w] = -INFINITY;
              if (g + 8 >= seen) acc[k][w + 2] = -INFINITY;
            }
        }
        bool rise = false;
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            rise |= fmaxf(acc[k][w], acc[k][w + 2]) > fminf(m[k][w], mv[k][w] + SHIFT - info.lv) + 8.0f;
            if constexpr (SCORES) {
              if (wq * 8 * NT + 8 * k + 2 * t4 + w < rows) {
                float *to = (ONE ? score[0][0] + (int64_t)(8 * k + w) * a.score_cols
                                 : score[ONE ? 0 : k][ONE ? 0 : w]) + t0;
                to[0] = acc[k][w];
                to[8] = acc[k][w + 2];
              }
            }
          }
        if (__any_sync(FULL, rise)) {
#pragma unroll
          for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              float top = fmaxf(acc[k][w], acc[k][w + 2]);
              for (int sh = 4; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, sh));
              const float mn = fmaxf(m[k][w], top), mvn = fmaxf(mv[k][w], top + info.lv - SHIFT);
              const float fl = exp2_fast(m[k][w] - mn), fo = exp2_fast(mv[k][w] - mvn);
              m[k][w] = mn;
              mv[k][w] = mvn;
              l[k][w] *= fl;
#pragma unroll
              for (int n = 0; n < MT; ++n) {
                o[k][n][w] *= fo;
                o[k][n][w + 2] *= fo;
              }
            }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int k = 0; k < NT; ++k) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            l[k][e & 1] += exp2_fast(acc[k][e] - m[k][e & 1]);
            p[e] = exp2_fast(acc[k][e] + (info.lv - mv[k][e & 1]));
          }
          pb[k][0] = transpose8(pack2<IBP_FP16>(p[0], p[1]));
          pb[k][1] = transpose8(pack2<IBP_FP16>(p[2], p[3]));
        }
        if constexpr (!EARLY) load_values();
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          const uint32_t u0 = code_bias<CODE>(v[0][w]), u1 = code_bias<CODE>(v[1][w]);
          const uint32_t u2 = code_bias<CODE>(v[2][w]), u3 = code_bias<CODE>(v[3][w]);
          const uint32_t p01 = __byte_perm(u0, u1, 0x5140), p23 = __byte_perm(u0, u1, 0x7362);
          const uint32_t q01 = __byte_perm(u2, u3, 0x5140), q23 = __byte_perm(u2, u3, 0x7362);
          const uint32_t a0 = code_pair<CODE, 0>(p01), a1 = code_pair<CODE, 1>(p01),
                         a2 = code_pair<CODE, 0>(q01), a3 = code_pair<CODE, 1>(q01);
          const uint32_t b0 = code_pair<CODE, 0>(p23), b1 = code_pair<CODE, 1>(p23),
                         b2 = code_pair<CODE, 0>(q23), b3 = code_pair<CODE, 1>(q23);
#pragma unroll
          for (int k = 0; k < NT; ++k) {
            mma16816(o[k][2 * w], a0, a1, a2, a3, pb[k][0], pb[k][1]);
            mma16816(o[k][2 * w + 1], b0, b1, b2, b3, pb[k][0], pb[k][1]);
          }
        }
      }
      if (tile == tile0 + count - 1) break;  // the last one's stage is kept for the join
      __syncwarp();
      if (lane == 0) mbar_arrive(&freed[s]);
      if (++s == ST) {
        s = 0;
        phase ^= 1u;
      }
    }

    // ---- join the warps' results of this stretch in the last tile's stage (its 2 * TILE *
    // D bytes hold 8 rows of every warp), then finish the segment or leave a part
    const bool first = x == lo, done = tile0 == 0 && count == nt;
    float *part = a.part + ((int64_t)cta * 2 + (first ? 0 : 1)) * S::part_floats;
    float *merge = reinterpret_cast<float *>(stages + s * S::stage_bytes);
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      consumer_sync();
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float sum = l[k][w];
        for (int sh = 4; sh < 32; sh <<= 1) sum += __shfl_xor_sync(FULL, sum, sh);
        const int at = warp * 8 + 2 * t4 + w;
        if (g == 0) {
          st_m[at] = m[k][w];
          st_mv[at] = mv[k][w];
          st_l[at] = sum;
        }
        // elements g*D/8 .. of the row, in 16-byte pieces that the row's number scatters
        float4 *to = reinterpret_cast<float4 *>(merge + at * D);
#pragma unroll
        for (int n = 0; n < MT / 2; ++n)
          to[(g * (D / 32) + n) ^ t4] = make_float4(o[k][2 * n][w], o[k][2 * n][w + 2],
                                                   o[k][2 * n + 1][w], o[k][2 * n + 1][w + 2]);
      }
      consumer_sync();
      for (int u = threadIdx.x; u < wqn * 8 * (D / 4); u += 32 * CONSUMERS) {
        const int in = u / (D / 4) % 8, side = u / (D / 4) / 8, piece = u % (D / 4);
        const int r = side * 8 * NT + 8 * k + in;
        if (r >= rows) continue;
        float top = NONE, topv = NONE;
        for (int i = 0; i < wkn; ++i) {
          const int at = (i * wqn + side) * 8 + in;
          top = fmaxf(top, st_m[at]);
          topv = fmaxf(topv, st_mv[at]);
        }
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float sum = 0.0f;
        for (int i = 0; i < wkn; ++i) {
          const int at = (i * wqn + side) * 8 + in;
          const float4 z = reinterpret_cast<const float4 *>(merge + at * D)[piece ^ (in >> 1)];
          const float f = exp2_fast(st_mv[at] - topv);
          y.x += z.x * f;
          y.y += z.y * f;
          y.z += z.z * f;
          y.w += z.w * f;
          sum += st_l[at] * exp2_fast(st_m[at] - top);
        }
        if (done) {
          const int rr = r0 + r;
          const int64_t row = sq.row0 + rr / group;
          const int qh = head * group + rr % group;
          const float f = sum > 0.0f ? exp2_fast(topv - top) / sum : 0.0f;
          *reinterpret_cast<uint2 *>(static_cast<char *>(a.q.out) +
                                     2 * (row * a.q.out_row_stride + qh * a.q.out_head_stride + 4 * piece)) =
              make_uint2(pack2<DT>(y.x * f, y.y * f), pack2<DT>(y.z * f, y.w * f));
          if (piece == 0) {
            const float z = sum > 0.0f ? top + log2f(sum) : -INFINITY;
            if (a.q.d_lse) a.q.d_lse[row * a.q.q_heads + qh] = z * LN2;
            if constexpr (SCORES) a.lse2[score_row(a, sq, b, head) + rr] = z;
          }
        } else {
          reinterpret_cast<float4 *>(part)[r * (D / 4) + piece] = y;
          if (piece == 0)
            reinterpret_cast<float4 *>(part + MB * D)[r] = make_float4(top, topv, sum, 0.0f);
        }
      }
    }
    consumer_sync();
    fence_async_proxy();
    __syncwarp();
    if (lane == 0) mbar_arrive(&freed[s]);
    if (++s == ST) {
      s = 0;
      phase ^= 1u;
    }
    x += count;
  }
}

// ---- host side -------------------------------------------------------------------

int score_cols_of(const ibp_kv_cache &c) {
  return (c.table_cols * c.page_tokens + TILE - 1) / TILE * TILE;
}

// Query rows of a segment: the fewest that hold a sequence's rows of one K/V head, so that
// its codes are read and converted for all of them at once (no more than 32 rows come here
// without weights). 64 sequences of 16,384 tokens, 8 heads of 128 elements: 16 rows 494 us,
// in segments of 8 662; 32 rows 840 us, in segments of 16 961.
int rows_of(int64_t max_rows) {
  return max_rows <= 8 ? 8 : max_rows <= 16 ? 16 : max_rows <= 32 ? 32 : 64;
}

// How many sequences and how many rows of each a launch is for. The scores that weights are
// added up from are held for those alone: at most SCORE_BYTES of them, or one row of one
// sequence. Where all rows of a call need more, it goes over them in slices, one after another,
// and adds each slice's probabilities to the weights that the one before left; sequences are
// divided before a slice gets fewer rows than a segment takes.
constexpr int64_t SCORE_BYTES = int64_t(1) << 30;
struct Portion {
  int batch, rows;     // rows 0: all of them
  int64_t score_rows;  // rows whose scores are held
};
Portion portion_of(const ibp_kv_cache &c, int64_t n_rows, int64_t max_q, int q_heads, bool weights) {
  if (!weights) return {MAX_BATCH, 0, 0};
  const int64_t row_bytes = std::max<int64_t>((int64_t)q_heads * score_cols_of(c) * sizeof(float), 1);
  const int64_t fit = std::max<int64_t>(SCORE_BYTES / row_bytes, 1);
  if (n_rows <= fit) return {MAX_BATCH, 0, n_rows};
  const int64_t group = q_heads / c.n_heads, whole = 64 / std::gcd<int64_t>(64, group);
  const int64_t least = std::min((64 + group - 1) / group, max_q);
  Portion y;
  y.batch = (int)std::min<int64_t>({std::max<int64_t>(fit / least, 1), c.batch, MAX_BATCH});
  int64_t rows = std::max<int64_t>(fit / y.batch, 1);
  if (rows > whole) rows -= rows % whole;  // whole segments of 64 rows
  y.rows = (int)std::min(rows, max_q);
  y.score_rows = (int64_t)y.batch * y.rows;
  return y;
}

struct Layout {
  size_t part, lse2, scores, bytes;
};
Layout layout_of(const ibp_kv_cache &c, const Portion &p, int64_t max_q, int q_heads) {
  const int mb = rows_of((p.rows ? p.rows : max_q) * (q_heads / c.n_heads));
  Layout y;
  y.part = 0;
  y.lse2 = y.part + (size_t)MAX_CTAS * 2 * mb * (c.head_dim + 4) * sizeof(float);
  y.scores = y.lse2 + ((size_t)p.score_rows * q_heads * sizeof(float) + 255) / 256 * 256;
  y.bytes = y.scores + (size_t)p.score_rows * q_heads * score_cols_of(c) * sizeof(float);
  return y;
}

// Query rows of a sequence that one launch is for, at most.
int64_t launch_rows_of(const AttentionArgs &a) { return a.slice_rows ? a.slice_rows : a.q.max_q; }

template <int D, int CODE, int DT, int NT, int WQ, bool SCORES>
int launch_shape(AttentionArgs a, const DeviceInfo &dev, cudaStream_t s) {
  using S = Shape<D, NT, WQ>;
  auto kernel = kv_attend_kernel<D, CODE, DT, NT, WQ, SCORES>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::smem) !=
      cudaSuccess)
    return IBP_ERR_CUDA;
  const int group = a.q.q_heads / a.c.n_heads;
  const int64_t blocks = (launch_rows_of(a) * group + S::MB - 1) / S::MB;
  const int64_t most = (int64_t)a.batch * a.c.n_heads * blocks * (a.score_cols / TILE);
  a.ctas = (int)std::min<int64_t>(std::min(S::per_sm * dev.sm_count, MAX_CTAS), std::max<int64_t>(most, 1));
  kernel<<<a.ctas, THREADS, S::smem, s>>>(a);
  if (cudaGetLastError() != cudaSuccess) return IBP_ERR_CUDA;
  const int64_t chunks = SCORES ? (a.score_cols + WEIGHT_TOKENS - 1) / WEIGHT_TOKENS : 0;
  if (launch_dependent(kv_finish_kernel<D, DT, typename S::Plan, SCORES>,
                       dim3((unsigned)(blocks + chunks), (unsigned)a.c.n_heads, (unsigned)a.batch),
                       dim3(FINISH_THREADS), 0, s, a, (int)blocks) != cudaSuccess)
    return IBP_ERR_CUDA;
  return IBP_OK;
}

template <int D, int CODE, int DT>
int launch_rows(const AttentionArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const bool w = a.q.d_weights != nullptr;
  switch (rows_of(launch_rows_of(a) * (a.q.q_heads / a.c.n_heads))) {
    case 8:
      return w ? launch_shape<D, CODE, DT, 1, 1, true>(a, dev, s)
               : launch_shape<D, CODE, DT, 1, 1, false>(a, dev, s);
    case 16:
      return w ? launch_shape<D, CODE, DT, 2, 1, true>(a, dev, s)
               : launch_shape<D, CODE, DT, 2, 1, false>(a, dev, s);
    case 32:
      return w ? launch_shape<D, CODE, DT, 2, 2, true>(a, dev, s)
               : launch_shape<D, CODE, DT, 2, 2, false>(a, dev, s);
    default: return launch_shape<D, CODE, DT, 2, 4, true>(a, dev, s);  // weights: see many_rows
  }
}

template <int D>
int launch_types(const AttentionArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  if (a.c.code == IBP_KV_INT8)
    return a.q.dtype == IBP_BF16 ? launch_rows<D, IBP_KV_INT8, IBP_BF16>(a, dev, s)
                                 : launch_rows<D, IBP_KV_INT8, IBP_FP16>(a, dev, s);
  return a.q.dtype == IBP_BF16 ? launch_rows<D, IBP_KV_E4M3, IBP_BF16>(a, dev, s)
                               : launch_rows<D, IBP_KV_E4M3, IBP_FP16>(a, dev, s);
}

}  // namespace

// More rows go to the kernel for many of them, which keeps no scores to add weights up from.
// (128 K/V heads over 4,096 tokens, 128 elements a head, this kernel against that one:
// 24 rows 84 us | 88, 32 rows 87 | 91, 64 rows 142 | 94, 128 rows 236 | 97.) Measured with equal
// counts; the largest count decides for the whole launch, so a chunk of a prompt takes
// decoding sequences along: 63 of 4,096 tokens with one row beside one with 512, 32 query heads
// on 8, take 323 us in one call and 117 + 85 in two.
static bool many_rows(const ibp_kv_cache &c, int64_t max_q, int q_heads, bool weights) {
  return !weights && max_q * (q_heads / c.n_heads) > 32;
}

size_t kv_attention_scratch_bytes(const ibp_kv_cache &c, int64_t n_rows, int64_t max_q,
                                  int q_heads, bool with_weights) {
  max_q = std::min(max_q, n_rows);
  if (many_rows(c, max_q, q_heads, with_weights)) return kv_prefill_scratch_bytes(c);
  return layout_of(c, portion_of(c, n_rows, max_q, q_heads, with_weights), max_q, q_heads).bytes;
}

int launch_kv_attention(const ibp_kv_cache &c, const ibp_kv_query &query, void *d_scratch,
                        int32_t *d_status, cudaStream_t s) {
  ibp_kv_query q = query;
  q.max_q = std::min(q.max_q, q.n_rows);  // what a sequence can have, however high the bound given
  if (many_rows(c, q.max_q, q.q_heads, q.d_weights != nullptr))
    return launch_kv_prefill(c, q, d_scratch, d_status, s);
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  const Portion p = portion_of(c, q.n_rows, q.max_q, q.q_heads, q.d_weights != nullptr);
  const Layout y = layout_of(c, p, q.max_q, q.q_heads);
  char *base = static_cast<char *>(d_scratch);
  AttentionArgs a;
  a.c = c;
  a.q = q;
  a.status = d_status;
  a.wait_ns = gather_wait_limit_ns();
  a.withhold = withhold_plans();
  a.score_cols = score_cols_of(c);
  a.part = reinterpret_cast<float *>(base + y.part);
  a.lse2 = reinterpret_cast<float *>(base + y.lse2);
  a.scores = q.d_weights ? reinterpret_cast<float *>(base + y.scores) : nullptr;
  a.slice_rows = p.rows;
  for (a.b0 = 0; a.b0 < c.batch; a.b0 += p.batch) {
    a.batch = std::min(c.batch - a.b0, p.batch);
    a.slice0 = 0;
    do {
      a.q.d_weights_in = a.slice0 ? q.d_weights : q.d_weights_in;
      a.q.decay = a.slice0 ? 1.0f : q.decay;
      if (int rc = c.head_dim == 64 ? launch_types<64>(a, dev, s) : launch_types<128>(a, dev, s))
        return rc;
      a.slice0 += p.rows;
    } while (p.rows && a.slice0 < q.max_q);
  }
  return IBP_OK;
}

}  // namespace ibp
