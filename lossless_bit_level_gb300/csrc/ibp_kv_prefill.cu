// Attention of many query rows over the 8-bit paged key/value cache, on the fifth
// generation's matrix unit (declared in include/ibp.h; the formulas stand at the head of
// ibp_kv_attend.cuh).
//
// A CTA takes 256 query rows of one K/V head (the rows of all query heads that share it,
// so shared heads fill the matrix unit) over tiles of 128 tokens. Codes become fp16 in
// shared memory, exactly, once for both halves of 128 rows; S = Q K^T and O += P V
// accumulate in tensor memory, P returns there as fp16. While the matrix unit works on
// one half, the other half's 128 threads (one to a row) turn scores into probabilities:
//   warps 0-3, 4-7  rows 0-127 and 128-255: references, exponentials, the final scaling
//   warps 8-11      convert codes, store them swizzled
//   warps 12, 14    issue the matrix instructions of a half each (one warp alone took 75
//                   cycles an instruction)
//   warp 13         looks up pages and scales, fetches codes with bulk copies two tiles ahead
//                   (15 only completes the warpgroup)
// A page's key scale is a factor of its scores, its value scale one of its probabilities.
//
// Bound by arithmetic: 4 D operations a (row, token) pair, and one exponential. Up to 2,048
// rows of 2 sequences of 5,001 to 8,192 tokens, 32 query heads on 8 of 128 elements (241
// GFLOP): 259 us with the joining, 929 TFLOP/s, half of what plain products reach. The
// matrix unit is busy 59 % of the time; what bounds it is the chain of a half tile (read scores,
// 64 exponentials a thread, store P, hand over: about 2,000 cycles for the two halves
// that take turns) and shared memory, which holds Q and both fp16 tiles. Places for scores
// of 128 tokens would need all of tensor memory; starting one half late was slower (282 us
// against 270). Two places for scores with P over them took 272 us with a wait for the product
// that reads P.
#include <algorithm>
#include <type_traits>

#include "ibp_kv_attention.cuh"

namespace ibp {

namespace {

constexpr int MB = 256;      // query rows of a segment
constexpr int TILE = 128;    // tokens of a tile
constexpr int GROUPS = TILE / 16;
constexpr int STAGES = 2;    // tiles of K in fp16, of K's codes and of V's codes
constexpr int V_HALVES = 2;  // half tiles of V in fp16
constexpr int INFOS = 8;     // tiles whose scales are kept
constexpr int BATCH = 128;   // sequences of one launch
constexpr int THREADS = 16 * 32;
// registers a thread, out of 128 each at launch: 8 * 168 + 4 * 88 + 4 * 88 = 16 * 128 a lane
constexpr int ROW_REGS = 168, CONVERT_REGS = 88, ISSUE_REGS = 88;
constexpr int CONVERT_WARP = 8, ISSUE_WARP = 12, FETCH_WARP = 13;
// Scores come 64 tokens (half a tile) at a time. Once a thread has read them into its registers
// the next ones may go over them, so that they are there when it is done; P goes to two places of
// its own in turn. No instruction writes what an earlier one may still read: matrix instructions
// of different accumulators need not run in the order of their issue. S at 128 w, P at
// 128 w + 64 + 32 (half), O at 256 + 128 w.
constexpr int HALF = 64;
constexpr uint32_t TMEM_COLS = 512, O_COL = 256;
// The largest factor of a row when its reference is set is 2^ROW_SHIFT (from a sum of 16
// factors: between that and 2^4 times it). Lower than SHIFT: here a row that outgrows its
// reference costs the whole warp (2048 rows over 8192 tokens: 306 us with 7, 277 with 4).
constexpr float ROW_SHIFT = 2.0f;
// SHARED spans are seen whole by all their rows. SPLIT (of SHARED): no more than 128 rows, which
// both halves of the CTA hold: half w takes the tiles of its stretch whose number has its parity,
// so that neither waits for the other and no half is without rows. Each half leaves results of
// its own, in the place of 128 rows each, and the joining adds them up.
template <bool SPLIT>
constexpr int ROWS_OF = SPLIT ? MB / 2 : MB;
template <Over OVER, bool SPLIT>
using PlanOf = std::conditional_t<OVER == Over::SHARED, EvenPlan<ROWS_OF<SPLIT>, TILE>, CausalPlan<MB, TILE>>;

// ---- tensor memory and the matrix instruction
__device__ __forceinline__ void tmem_alloc(uint32_t *at) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(at)),
               "r"(TMEM_COLS)
               : "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base) {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(TMEM_COLS));
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// One lane of the warp, the same every time; the matrix instructions are issued by it while
// the whole warp computes their operands (uniform over the warp, so in uniform registers).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e;
}
// The barrier is arrived at once every matrix instruction issued so far has finished.
__device__ __forceinline__ void tc_commit(uint64_t *bar, uint32_t mine) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(
          smem_u32(bar)),
      "r"(mine)
      : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add,
                                       uint32_t mine) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add), "r"(mine)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add,
                                       uint32_t mine) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add), "r"(mine)
      : "memory");
}

#define R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), \
                 "=r"(x[i + 5]), "=r"(x[i + 6]), "=r"(x[i + 7])
#define I8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), \
                 "r"(x[i + 5]), "r"(x[i + 6]), "r"(x[i + 7])

// Columns of this warp's 32 lanes, a lane to a thread, loaded and waited for in one statement:
// nothing may copy a register in between.
__device__ __forceinline__ void tmem_read64(uint32_t at, uint32_t *x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
      " tcgen05.wait::ld.sync.aligned;"
      : R8(x, 0), R8(x, 8), R8(x, 16), R8(x, 24), R8(x, 32), R8(x, 40), R8(x, 48), R8(x, 56)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_read32(uint32_t at, uint32_t *x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      " tcgen05.wait::ld.sync.aligned;"
      : R8(x, 0), R8(x, 8), R8(x, 16), R8(x, 24)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_read16(uint32_t at, uint32_t *x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      " tcgen05.wait::ld.sync.aligned;"
      : R8(x, 0), R8(x, 8)
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t *x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16};" ::"r"(at),
      I8(x, 0), I8(x, 8)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_store() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Shared-memory operand in 128-byte rows of 64 fp16, swizzled in groups of 8 rows.
// K-major (the summed index along the row): groups of 8 rows 1024 bytes apart. MN-major
// (the summed index down the rows): the same 1024 bytes between groups of 8 of the summed
// index, `block` bytes between blocks of 64 of the other.
// (The descriptor's upper half is the same for all; `offset` bytes are added to the start.)
__device__ __forceinline__ uint32_t operand(const void *p, uint32_t block) {
  return (smem_u32(p) >> 4) | ((block >> 4) << 16);
}
__device__ __forceinline__ uint64_t operand_at(uint32_t base, uint32_t offset) {
  constexpr uint32_t upper = (1024 >> 4) | (1u << 14) | (2u << 29);
  return ((uint64_t)upper << 32) | (base + (offset >> 4));
}
// fp16 operands, fp32 accumulators, 128 rows, n columns; vt: the second operand MN-major.
__host__ __device__ constexpr uint32_t instruction(int n, bool vt) {
  return (1u << 4) | ((vt ? 1u : 0u) << 16) | ((uint32_t)(n / 8) << 17) | ((uint32_t)(128 / 16) << 24);
}

// Scales of a tile's groups of 16 tokens (a group never spans two pages); bad: a bit for
// each group whose page is not there; held: tokens of the tile that the sequence has.
struct TileInfo {
  float2 scale[GROUPS];  // key scale, log2 of the value scale
  uint32_t bad;
  int held;
};

template <int D>
struct Memory {
  static constexpr int q_bytes = 128 * D * 2, kv_bytes = TILE * D * 2, half_bytes = HALF * D * 2;
  static constexpr int code_bytes = TILE * D;
  static constexpr int q = 0, k = 2 * q_bytes, v = k + STAGES * kv_bytes, raw_k = v + V_HALVES * half_bytes,
                       raw_v = raw_k + STAGES * code_bytes;
  static constexpr int info = raw_v + STAGES * code_bytes, bars = info + INFOS * (int)sizeof(TileInfo);
  static constexpr int barriers = 38 + INFOS;  // see the kernel's list of them
  static constexpr int prefix = bars + barriers * 8;
  static constexpr int cursors = (prefix + (BATCH + 1) * 8 + 15) / 16 * 16;
  static constexpr int words = cursors + 9 * 48;
  static constexpr int bytes = words + 16;
};

// Where a stretch stands: the segment of tile x and the tile within it. Each warp keeps
// its own in shared memory, out of the registers of its inner loop.
struct __align__(16) Cursor {
  int b, head, block, tile, tiles;
  Sequence seq;
};
template <Over OVER, bool SPLIT>
__device__ __forceinline__ Cursor cursor_at(const AttentionArgs &a, const int64_t *prefix, int group,
                                            int64_t x) {
  Cursor c;
  c.b = find_sequence(prefix, a.batch, x);
  c.seq = sequence_of<OVER>(a, c.b, nullptr);
  const PlanOf<OVER, SPLIT> plan(c.seq, group);
  if constexpr (OVER == Over::SHARED)
    if (((x | prefix[c.b + 1]) >> 31) == 0) {  // divisions in 32 bits take a fraction of the time
      const uint32_t local = (uint32_t)(x - prefix[c.b]), segment = local / (uint32_t)plan.tiles_each;
      c.head = (int)(segment / (uint32_t)plan.blocks);
      c.block = (int)segment - c.head * plan.blocks;
      c.tile = (int)(local - segment * (uint32_t)plan.tiles_each);
      c.tiles = plan.tiles_each;
      return c;
    }
  const int64_t local = x - prefix[c.b], per_head = (prefix[c.b + 1] - prefix[c.b]) / a.c.n_heads;
  c.head = (int)(local / per_head);
  const int64_t in = local - c.head * per_head;
  c.block = plan.find(in);
  c.tile = (int)(in - plan.before(c.block));
  c.tiles = plan.tiles(c.block);
  return c;
}
static_assert(sizeof(Cursor) <= 48, "the place kept for it");
// The first tile of the next segment that has one (there is one: the caller's x < total).
template <Over OVER, bool SPLIT>
__device__ __forceinline__ void next_segment(const AttentionArgs &a, const int64_t *prefix, int group,
                                             Cursor &c) {
  c.tile = 0;
  for (;;) {
    const PlanOf<OVER, SPLIT> plan(c.seq, group);
    if (++c.block == plan.blocks) {
      c.block = 0;
      if (++c.head == a.c.n_heads) {
        c.head = 0;
        do {
          ++c.b;
        } while (prefix[c.b] == prefix[c.b + 1]);
        c.seq = sequence_of<OVER>(a, c.b, nullptr);
      }
    }
    c.tiles = PlanOf<OVER, SPLIT>(c.seq, group).tiles(c.block);
    if (c.tiles > 0) return;
  }
}

// Codes to fp16, exactly (as in ibp_kv_attend.cuh).
template <int CODE, int HIGH>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  if constexpr (CODE == IBP_KV_INT8) {
    const uint32_t u = __byte_perm(w ^ 0x80808080u, 0x64646464u, HIGH ? 0x4342 : 0x4140);
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&u), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&h);
  } else {
    uint32_t y;
    const uint16_t x = HIGH ? (uint16_t)(w >> 16) : (uint16_t)w;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(x));
    return y;
  }
}

template <int D, int CODE, int DT, Over OVER, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1) kv_prefill_kernel(const __grid_constant__ AttentionArgs a) {
  using M = Memory<D>;
  using Plan = PlanOf<OVER, SPLIT>;
  static_assert(M::info % alignof(TileInfo) == 0 && M::bars % 8 == 0 && M::prefix % 8 == 0 &&
                    M::cursors % alignof(Cursor) == 0 && M::words % 8 == 0 && M::bytes <= 227 * 1024,
                "what lies in shared memory is aligned and fits");
  extern __shared__ __align__(1024) unsigned char smem[];
  TileInfo *info = reinterpret_cast<TileInfo *>(smem + M::info);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + M::bars);
  uint64_t *k_full = bars, *k_free = bars + 2, *raw_k_full = bars + 4, *raw_k_free = bars + 6,
           *q_full = bars + 8, *last = bars + 10, *raw_v_full = bars + 12, *raw_v_free = bars + 14,
           *v_full = bars + 16, *v_free = bars + 18;
  // [2 w + half]: a row's thread may be two instructions ahead of the last one done
  uint64_t *s_full = bars + 20, *p_full = bars + 24, *o_done = bars + 28, *s_free = bars + 32,
           *info_full = bars + 36;
  // SPLIT: a half's tiles have their own (it would not tell the phases of the other's apart)
  auto v_full_of = [&](int tile, int half) {
    return SPLIT && (tile & 1) ? bars + 36 + INFOS + half : v_full + half;
  };
  int64_t *prefix = reinterpret_cast<int64_t *>(smem + M::prefix);
  uint32_t *tmem_at = reinterpret_cast<uint32_t *>(smem + M::words);
  volatile int *abort = reinterpret_cast<volatile int *>(smem + M::words + 4);

  constexpr int STEP = SPLIT ? 2 : 1;  // between tiles of a half
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
  const ibp_kv_cache &c = a.c;
  const int group = a.q.q_heads / c.n_heads;
  if constexpr (OVER == Over::ALL) grid_launch_dependents();
  if (smem_u32(smem) & 1023) {  // the operands' rows would be swizzled otherwise than written
    report(a.status, IBP_ERR_CUDA);
    if (OVER == Over::ALL && threadIdx.x == 0) a.cuts[cta] = Cut();
    if constexpr (OVER == Over::SHARED) grid_dependency_wait();
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&k_free[i], SPLIT ? 1 : 2);
      mbar_init(&raw_k_full[i], 1);
      mbar_init(&raw_k_free[i], 4);
      mbar_init(&raw_v_full[i], 1);
      mbar_init(&raw_v_free[i], 4);
      mbar_init(v_full_of(0, i), 4);
      mbar_init(&v_free[i], SPLIT ? 1 : 2);
      mbar_init(v_full_of(1, i), 4);
      mbar_init(&q_full[i], 4);
      mbar_init(&last[i], 1);
    }
    for (int i = 0; i < INFOS; ++i) mbar_init(&info_full[i], 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_free[i], 4);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    *abort = 0;
    mbar_init_fence();
  }
  if constexpr (OVER == Over::SHARED) {
    grid_dependency_wait();  // the spans
    grid_launch_dependents();  // they are there for the next grid too
    if (cta >= ctas_of<OVER>(a)) return;  // the SM is for that one
  }
  if (warp == ISSUE_WARP) {
    tmem_alloc(tmem_at);
    int64_t base = 0;
    for (int k0 = 0; k0 < a.batch; k0 += 32) {
      const int b = k0 + lane;
      int64_t tiles = 0;
      if (b < a.batch) {
        const Plan plan(sequence_of<OVER>(a, b, cta == 0 ? a.status : nullptr), group);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  const Split split(prefix[a.batch], ctas_of<OVER>(a));
  const bool work = cta < split.ctas;
  const int64_t lo = work ? split.start(cta) : 0, hi = work ? split.start(cta + 1) : 0;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (mbar_wait(bar, parity, abort, a.wait_ns)) return true;
    report(a.status, IBP_ERR_TIMEOUT);
    *abort = 1;
    return false;
  };

  if (warp >= CONVERT_WARP && warp < ISSUE_WARP) {
    fewer_registers<CONVERT_REGS>();
    if (work) {
    // ---- codes to fp16, half a tile at a time: a thread takes 16 elements of every STEP-th
    // token. Rows of tokens, 64 elements to a 128-byte row, the 16-byte pieces of a row
    // exclusive-or'ed with its number (which is the same for all of a thread's tokens). At
    // 128 elements, 16 threads take two tokens, the second four of each eight those of the
    // other token: then neither the loads nor the stores of eight threads share a bank.
    constexpr int PER = D / 16, STEP = 128 / PER, N = HALF / STEP;  // 8, 16, 4 or 4, 32, 2
    const int tid = threadIdx.x - CONVERT_WARP * 32;
    const int piece = D == 128 ? tid & 7 : tid & 3;
    const int key0 = D == 128 ? 2 * (tid >> 4) + (((tid >> 3) ^ (tid >> 2)) & 1) : tid >> 2;
    const int n = (int)(hi - lo);
    const int from = key0 * D + piece * 16, block = (2 * piece) / 8;
    int to[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) to[h] = key0 * 128 + (((2 * piece + h) ^ key0) & 7) * 16;
    int held = 0;
    uint32_t bad = 0;
    auto load = [&](uint4 *w, const unsigned char *raw, int half) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint4 *>(raw + from + i * (STEP * D));
      if (held < TILE || bad) {  // what no page gave is not a number of ours
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int key = half * HALF + key0 + i * STEP;
          if (key >= held || ((bad >> (key / 16)) & 1)) w[i] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    };
    auto store = [&](const uint4 *w, unsigned char *out) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<uint4 *>(out + to[h] + i * (STEP * 128)) =
              make_uint4(code_pair<CODE, 0>(u[2 * h]), code_pair<CODE, 1>(u[2 * h]),
                         code_pair<CODE, 0>(u[2 * h + 1]), code_pair<CODE, 1>(u[2 * h + 1]));
      }
    };
    auto ready = [&](uint64_t *bar, uint32_t parity) { return __all_sync(FULL, wait(bar, parity)); };
    auto done = [&](uint64_t *bar, uint64_t *raw_bar) {
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar);
        if (raw_bar) mbar_arrive(raw_bar);
      }
    };
    // K of tile 0, then K of tile g + 1 before V of tile g: the scores of a tile are wanted
    // a tile before its values
#pragma unroll 1
    for (int g = -1; g < n; ++g) {
      if (g + 1 < n) {
        const int s = (g + 1) & 1;
        const uint32_t turn = (uint32_t)((g + 1) >> 1) & 1;
        if (!ready(&raw_k_full[s], turn) || (g + 1 >= STAGES && !ready(&k_free[s], turn ^ 1u))) break;
        held = info[(g + 1) & (INFOS - 1)].held;
        bad = info[(g + 1) & (INFOS - 1)].bad;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint4 w[N];
          load(w, smem + M::raw_k + s * M::code_bytes + half * (HALF * D), half);
          store(w, smem + M::k + s * M::kv_bytes + block * (TILE * 128) + half * (HALF * 128));
        }
        done(&k_full[s], &raw_k_free[s]);
      }
      if (g >= 0) {
        const int s = g & 1;
        held = info[g & (INFOS - 1)].held;
        bad = info[g & (INFOS - 1)].bad;
        bool ok = ready(&raw_v_full[s], (uint32_t)(g >> 1) & 1);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (g >= 1) ok = ok && ready(&v_free[half], (uint32_t)(g - 1) & 1);
          if (!ok) break;
          uint4 w[N];
          load(w, smem + M::raw_v + s * M::code_bytes + half * (HALF * D), half);
          store(w, smem + M::v + half * M::half_bytes + block * (HALF * 128));
          done(v_full_of(g, half), half ? &raw_v_free[s] : nullptr);
        }
        if (!ok) break;
      }
    }
    }
  } else if (warp >= ISSUE_WARP) {
    fewer_registers<ISSUE_REGS>();
    if (work && (warp == ISSUE_WARP || warp == ISSUE_WARP + 2)) {
      constexpr uint32_t is = instruction(HALF, false), io = instruction(D, true);
      const int w = (warp - ISSUE_WARP) / 2;
      const uint32_t mine = elect_one(), s_at = tmem + 128 * w, o_at = tmem + O_COL + 128 * w;
      const uint32_t q_at = operand(smem + M::q + w * M::q_bytes, 16), k_at = operand(smem + M::k, 16),
                     v_at = operand(smem + M::v, HALF * 128);
      auto ready = [&](uint64_t *bar, uint32_t parity) { return __all_sync(FULL, wait(bar, parity)); };
      // half h of the tile whose K is in stage s
      auto scores = [&](uint32_t s, int h) {
        const uint32_t k = k_at + s * (M::kv_bytes >> 4) + h * (HALF * 128 >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ss(s_at, operand_at(q_at, (i / 4) * (128 * 128) + (i % 4) * 32),
                 operand_at(k, (i / 4) * (TILE * 128) + (i % 4) * 32), is, i > 0, mine);
        tc_commit(&s_full[2 * w + h], mine);
        if (h) tc_commit(&k_free[s], mine);
      };
      Cursor cur = cursor_at<OVER, SPLIT>(a, prefix, group, lo);
      const int n = (int)(hi - lo);
      int g = 0;  // tiles of the stretch begun
      uint32_t segment = 0;
      bool ok = true;
      while (ok && g < n) {
        const int count = min(cur.tiles - cur.tile, n - g);
        const int skip = SPLIT ? (g ^ w) & 1 : 0, mine_of = SPLIT ? (count - skip + 1) / 2 : count;
        int x = g + skip;  // the half's own tiles: every STEP-th from here
        g += count;
        if (mine_of > 0) {
          ok = ready(&k_full[x & 1], (x >> 1) & 1) && ready(&q_full[w], segment & 1);
          if (!ok) break;
          tc_fence_after();
          scores(x & 1, 0);
          for (int j = 0; j < mine_of && ok; ++j, x += STEP) {
            const uint32_t turn = SPLIT ? (x >> 1) & 1 : x & 1;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if (h == 0 || j + 1 < mine_of) {  // the scores after these, once these have been read
                const int next = x + h * STEP;
                if (h) ok = ready(&k_full[next & 1], (next >> 1) & 1);
                ok = ok && ready(&s_free[2 * w + h], turn);
                if (!ok) break;
                tc_fence_after();
                scores(next & 1, h ^ 1);
              }
              ok = ready(v_full_of(x, h), turn) && ready(&p_full[2 * w + h], turn);
              if (!ok) break;
              tc_fence_after();
              const uint32_t v = v_at + h * (M::half_bytes >> 4), first = j > 0 || h > 0;
#pragma unroll
              for (int e = 0; e < HALF / 16; ++e)
                mma_ts(o_at, s_at + HALF + 32 * h + 8 * e, operand_at(v, e * 2048), io, e > 0 ? 1u : first,
                       mine);
              tc_commit(&o_done[2 * w + h], mine);
              tc_commit(&v_free[h], mine);
            }
          }
          ++segment;
        }
        if (ok && g < n) next_segment<OVER, SPLIT>(a, prefix, group, cur);
      }
      // nothing may be left running when this CTA gives its memory back
      tc_commit(&last[w], mine);
      drain(&last[w], 0, a.status);
      __syncwarp();
    }
    if (work && warp == FETCH_WARP) {
      // ---- a bulk copy for each part of a page that lies in the tile
      const int PP = min(c.page_tokens, TILE), n = (int)(hi - lo);
      const char *kc = static_cast<const char *>(c.k_codes), *vc = static_cast<const char *>(c.v_codes);
      struct Place {
        int b, head, t0, len;
      };
      Cursor *cur = reinterpret_cast<Cursor *>(smem + M::cursors) + 8;  // one for all lanes
      if (lane == 0) *cur = cursor_at<OVER, SPLIT>(a, prefix, group, lo);
      __syncwarp();
      int ahead = 0;  // tiles of the stretch taken
      auto take = [&] {
        const Place p = {cur->b, cur->head, cur->tile * TILE, cur->seq.len};
        ++ahead;
        __syncwarp();
        if (lane == 0 && ++cur->tile == cur->tiles && ahead < n) next_segment<OVER, SPLIT>(a, prefix, group, *cur);
        __syncwarp();
        return p;
      };
      // Lane g < 8 looks up the page of tokens 16 g .. : its id is asked for two tiles before
      // its codes, its scales one tile before.
      struct Pages {
        int page;
        float ks, vs;
      };
      auto ask = [&](const Place &p) {
        const int t = p.t0 + (lane & 7) * 16;
        if constexpr (OVER == Over::SHARED)
          return t < p.len ? __ldg(c.d_table + __ldcg(&a.spans[a.b0 + p.b].table_at) + t / c.page_tokens) : -1;
        return t < p.len ? __ldg(c.d_table + (int64_t)(a.b0 + p.b) * c.table_stride + t / c.page_tokens) : -1;
      };
      auto look_up = [&](const Place &p, int page) {
        Pages y = {-1, 0.0f, 0.0f};
        if (p.t0 + (lane & 7) * 16 < p.len) {
          if (page >= 0 && page < c.n_pages) {
            const int64_t at = (int64_t)page * c.n_heads + p.head;
            y.page = page;
            y.ks = __ldg(c.k_scales + at);
            y.vs = __ldg(c.v_scales + at);
          } else {
            report(a.status, IBP_ERR_INDEX);
          }
        }
        return y;
      };
      // The first tile's keys are asked for before anything of the second is looked up.
      Place now = take(), next = now, after = now;  // tiles g, g + 1 and g + 2
      const int first_page = ask(now);
      int next_page = -1, asked = -1;
      if (n > 1) {
        next = take();
        next_page = ask(next);
      }
      Pages py = look_up(now, first_page), ny = py;
      auto copy = [&](const char *codes, const Place &p, const Pages &y, unsigned char *to, uint64_t *bar) {
        const bool starts = lane < GROUPS && (lane * 16) % PP == 0 && y.page >= 0;
        const unsigned copies = __ballot_sync(FULL, starts);
        if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(__popc(copies) * PP * D));
        __syncwarp();
        if (starts)
          bulk_load(to + lane * 16 * D,
                    codes + kv_tile(c, y.page, p.head) +
                        (int64_t)((p.t0 + lane * 16) & (c.page_tokens - 1)) * D,
                    PP * D, bar);
      };
      auto fetch_k = [&](int g, const Place &p, const Pages &y) {
        const int s = g & 1;
        if (g >= STAGES &&
            !__all_sync(FULL, wait(&raw_k_free[s], (uint32_t)((g >> 1) & 1) ^ 1u)))
          return false;
        TileInfo &t = info[g & (INFOS - 1)];
        const unsigned bad = __ballot_sync(FULL, lane < GROUPS && y.page < 0);
        if (lane < GROUPS) t.scale[lane] = make_float2(y.ks, log2f(y.vs));
        if (lane == 0) {
          t.bad = bad;
          t.held = min(p.len - p.t0, TILE);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&info_full[g & (INFOS - 1)]);
        copy(kc, p, y, smem + M::raw_k + s * M::code_bytes, &raw_k_full[s]);
        return true;
      };
      int k_sent = 0, v_sent = 0;
      bool ok = fetch_k(0, now, py);
      k_sent = ok;
      if (n > 1) ny = look_up(next, next_page);
      if (n > 2) {
        after = take();
        asked = ask(after);
      }
      const int upto = a.withhold ? 1 : n;
      for (int g = 0; g < upto && ok; ++g) {
        if (g + 1 < n) {
          ok = fetch_k(g + 1, next, ny);
          if (!ok) break;
          k_sent = g + 2;
        }
        const int s = g & 1;
        if (g >= STAGES) ok = __all_sync(FULL, wait(&raw_v_free[s], (uint32_t)((g >> 1) & 1) ^ 1u));
        if (!ok) break;
        copy(vc, now, py, smem + M::raw_v + s * M::code_bytes, &raw_v_full[s]);
        v_sent = g + 1;
        now = next;
        next = after;
        py = ny;
        if (g + 2 < n) ny = look_up(next, asked);
        if (g + 3 < n) {
          after = take();
          asked = ask(after);
        }
      }
      // no copy may land after this CTA is gone, and the others may have stopped waiting for them
#pragma unroll 1
      for (int i = 0; i < 2 * STAGES; ++i) {
        const int k = (i < STAGES ? k_sent : v_sent) - 1 - i % STAGES;
        if (k >= 0)
          drain((i < STAGES ? raw_k_full : raw_v_full) + (k & 1), (uint32_t)((k >> 1) & 1), a.status);
      }
    }
    __syncwarp();
  } else {
    more_registers<ROW_REGS>();
    if (work) {
      // ---- one thread to a row
      const int w = warp >> 2, row = threadIdx.x & 127;
      const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
      const uint32_t sp = tmem + 128 * w + lanes, op = tmem + O_COL + 128 * w + lanes;
      unsigned char *q_to = smem + M::q + w * M::q_bytes + row * 128;
      Cursor *cur = reinterpret_cast<Cursor *>(smem + M::cursors) + warp;
      if (lane == 0) *cur = cursor_at<OVER, SPLIT>(a, prefix, group, lo);
      __syncwarp();
      if (OVER == Over::ALL && threadIdx.x == 0) {
        const Cut cut = {prefix[a.batch], cur->b, cur->head, cur->block, cur->tile, cur->tiles, 0};
        a.cuts[cta] = cut;
      }
      const int n_tiles = (int)(hi - lo), r = w * 128 + row;
      int x = 0;  // tiles of the stretch done
      bool ok = true;
      while (ok && x < n_tiles) {
        const int tile0 = cur->tile, count = min(cur->tiles - tile0, n_tiles - x);
        const int skip = SPLIT ? (x ^ w) & 1 : 0, mine_of = SPLIT ? (count - skip + 1) / 2 : count;
        const int rr = cur->block * ROWS_OF<SPLIT> + (SPLIT ? row : r);
        const bool live = rr < cur->seq.n * group;
        // the row in fp16, brought to a largest magnitude in [1, 2) by a power of two (bf16);
        // the sign of the scale goes with it, so that factors of scores are never negative
        float rowc = 0.0f;
        if (!SPLIT || mine_of > 0) {
          const char *src = static_cast<const char *>(a.q.q) +
                            2 * ((cur->seq.row0 + rr / group) * a.q.q_row_stride +
                                 (cur->head * group + rr % group) * a.q.q_head_stride);
          Raw16<DT> y[D / 16];
          uint32_t most = 0;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            y[i].clear();
            if (live) y[i].load(src + 32 * i);
          }
          float up = a.q.scale < 0.0f ? -1.0f : 1.0f, down = 1.0f;
          if constexpr (DT == IBP_BF16) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) most = y[i].largest(most);
            const int e = min(max((int)(Raw16<DT>::fold(most) >> 7) - 127, -120), 120);
            up *= __uint_as_float((uint32_t)(127 - e) << 23);
            down = __uint_as_float((uint32_t)(127 + e) << 23);
          }
          rowc = down * (fabsf(a.q.scale) * LOG2E);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float f[4];
              y[i].four(k, f);
              v[2 * k] = pack2<IBP_FP16>(f[0] * up, f[1] * up);
              v[2 * k + 1] = pack2<IBP_FP16>(f[2] * up, f[3] * up);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int at = 2 * i + h;
              *reinterpret_cast<uint4 *>(q_to + (at / 8) * (128 * 128) + ((at ^ row) & 7) * 16) =
                  make_uint4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
            }
          }
          fence_async_proxy();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full[w]);
        }
        const int limit = !live ? 0x7FFFFFFF
                          : OVER == Over::SHARED ? cur->seq.len
                                                 : max(cur->seq.len - cur->seq.n + rr / group + 1, 0);
        float m = NONE, mv = NONE, over = 0.0f;  // over: what the references are to rise by,
        bool pending = false;                     // if any row's are
        uint64_t l = 0;                           // two halves of the sum
        auto rescale = [&](float by, int before) {  // the output so far, once instruction `before` is done
          ok = __all_sync(FULL, wait(&o_done[2 * w + (before & 1)], (uint32_t)(before >> 1) & 1));
          if (!ok) return;
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) {
            uint32_t y[16];
            tmem_read16(op + 16 * k, y);
#pragma unroll
            for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * by);
            tmem_store16(op + 16 * k, y);
          }
          tmem_wait_store();
        };
#pragma unroll 1
        for (int j = 0; j < 2 * mine_of; ++j) {
          const int at_tile = skip + (j >> 1) * STEP, g = x + at_tile, h = j & 1;  // of the segment, the stretch; its half
          const int done_of = SPLIT ? g >> 1 : g, u = 2 * done_of + h;  // own tiles before, halves of tiles
          ok = __all_sync(FULL, (h || wait(&info_full[g & (INFOS - 1)], (uint32_t)((g / INFOS) & 1))) &&
                                    wait(&s_full[2 * w + h], (uint32_t)(done_of & 1)));
          if (!ok) break;
          tc_fence_after();
          const float2 *scale = info[g & (INFOS - 1)].scale + 4 * h;
          const uint32_t bad = (info[g & (INFOS - 1)].bad >> (4 * h)) & 15u;
          const int seen = limit - (tile0 + at_tile) * TILE - h * HALF;  // columns this row sees
          uint32_t s[HALF], p[HALF / 2];
          tmem_read64(sp, s);
          tc_fence_before();
          __syncwarp();
          if (elect_one()) mbar_arrive(&s_free[2 * w + h]);
          if (pending) {
            const float by = exp2_fast(-over);
            rescale(by, u - 1);
            if (!ok) break;
            m += over;
            mv += over;
            l = mul2(l, pair(by, by));
          }
          // With the references as they are: a probability with its value scale is
          // 2^(x + lv - mv), and the probability itself that times 2^(mv - m - lv), so one
          // exponential a score and one a group for the sum. It stands if every row has a
          // reference, sees all 64 tokens, has no value scale so small that the first could
          // vanish with the second still counting, and nothing passed fp16's range.
          uint64_t sum_l = l;
          // the largest sum of a group: no probability in it is larger
          float most = seen >= HALF && bad == 0 ? 0.0f : INFINITY;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 sc = scale[k];
            const float f = rowc * sc.x, up = sc.y - mv;
            const uint64_t ff = pair(f, f), uu = pair(up, up);
            uint64_t sum = 0;
#pragma unroll
            for (int e = 16 * k; e < 16 * k + 16; e += 2) {
              const uint64_t y = fma2(pair(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), ff, uu);
              const float p0 = exp2_fast(low(y)), p1 = exp2_fast(high(y));
              sum = add2(sum, pair(p0, p1));
              p[e / 2] = pack2<IBP_FP16>(p0, p1);
            }
            const float back = exp2_fast(-(sc.y + (m - mv)));
            sum_l = fma2(sum, pair(back, back), sum_l);
            most = fmaxf(most, fmaxf(low(sum) + high(sum), back <= 0x1p60f ? 0.0f : INFINITY));
          }
          // (a row of NaN has no largest sum and stands; its output is NaN either way)
          const uint32_t top = __reduce_max_sync(FULL, __float_as_uint(most));
          const bool stands = top <= __float_as_uint(32768.0f);
          pending = stands && top > __float_as_uint(16384.0f);
          if (stands) l = sum_l;
          if (pending) over = most > 16384.0f ? log2f(most) - (4.0f + ROW_SHIFT) : 0.0f;
          if (!stands) {  // masks, new references, then both exponents apart
            float mn = m, mvn = mv;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int n = (bad >> k) & 1 ? 0 : seen - 16 * k;
              float top = -INFINITY;
#pragma unroll
              for (int e = 0; e < 16; ++e) top = e < n ? fmaxf(top, __uint_as_float(s[16 * k + e])) : top;
              // (a masked group's -inf times a scale of zero is not a number: not a maximum either)
              top *= rowc * scale[k].x;
              mn = fmaxf(mn, top);
              mvn = fmaxf(mvn, top + scale[k].y - ROW_SHIFT);
            }
            if (__any_sync(FULL, mn > m + 8.0f || mvn > mv + 8.0f)) {
              const float fl = exp2_fast(m - mn), fo = exp2_fast(mv - mvn);
              m = mn;
              mv = mvn;
              l = mul2(l, pair(fl, fl));
              if (j > 0) {
                rescale(fo, u - 1);
                if (!ok) break;
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float f = rowc * scale[k].x, gv = exp2_fast(fminf(scale[k].y + (m - mv), 120.0f));
              const int n = (bad >> k) & 1 ? 0 : seen - 16 * k;
              float sum = 0.0f;
#pragma unroll
              for (int e = 0; e < 16; e += 2) {
                float p0 = exp2_fast(fmaf(__uint_as_float(s[16 * k + e]), f, -m));
                float p1 = exp2_fast(fmaf(__uint_as_float(s[16 * k + e + 1]), f, -m));
                p0 = e < n ? p0 : 0.0f;
                p1 = e + 1 < n ? p1 : 0.0f;
                sum += p0 + p1;
                p[8 * k + e / 2] = pack2<IBP_FP16>(p0 * gv, p1 * gv);
              }
              l = add2(l, pair(sum, 0.0f));
            }
          }
          const uint32_t at = sp + HALF + 32 * h;  // (the product before the last has read it:
          tmem_store16(at, p);                     // these scores were committed behind it)
          tmem_store16(at + 16, p + 16);
          tmem_wait_store();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * w + h]);
        }
        if (!ok) break;
        // ---- finish the segment, or leave a part
        const bool some = !SPLIT || mine_of > 0;
        if (some) {
          const int end = x + skip + (mine_of - 1) * STEP;  // the last of the half's tiles
          ok = __all_sync(FULL, wait(&o_done[2 * w + 1], (uint32_t)(SPLIT ? end >> 1 : end) & 1));
          if (!ok) break;
          tc_fence_after();
        }
        const float sum = low(l) + high(l);
        const bool done = tile0 == 0 && count == cur->tiles;
        const int64_t q_row = cur->seq.row0 + rr / group;
        const int q_head = cur->head * group + rr % group;
        float *part = a.part + ((int64_t)cta * 2 + (x == 0 ? 0 : 1)) * ((int64_t)MB * (D + 4));
        const float f = !done ? 1.0f : sum > 0.0f ? exp2_fast(mv - m) / sum : 0.0f;
        char *out = static_cast<char *>(a.q.out) +
                    2 * (q_row * a.q.out_row_stride + q_head * a.q.out_head_stride);
#pragma unroll 1
        for (int q4 = 0; q4 < D / 32; ++q4) {
          uint32_t s[32];
          tmem_read32(op + 32 * q4, s);
          if (!live) continue;
          float y[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = some ? __uint_as_float(s[e]) * f : 0.0f;
          if (OVER == Over::SHARED && done) {  // joined with the rows' other span later
            const int64_t at = q_row * a.q.q_heads + q_head + (SPLIT && w ? 2 * a.side_rows : 0);
            float4 *side = reinterpret_cast<float4 *>(a.side + at * D + 32 * q4);
#pragma unroll
            for (int e = 0; e < 8; ++e) side[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
          } else if (done) {
            store16<DT>(out + 64 * q4, y);
            store16<DT>(out + 64 * q4 + 32, y + 16);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4 *>(part + r * D + 32 * q4 + e) =
                  make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
        }
        tc_fence_before();
        if (live) {
          if (OVER == Over::SHARED && done) {
            a.side_lse2[q_row * a.q.q_heads + q_head + (SPLIT && w ? 2 * a.side_rows : 0)] = sum > 0.0f ? m + log2f(sum) : -INFINITY;
          } else if (done) {
            if (a.q.d_lse)
              a.q.d_lse[q_row * a.q.q_heads + q_head] = sum > 0.0f ? (m + log2f(sum)) * LN2 : -INFINITY;
          } else {
            reinterpret_cast<float4 *>(part + MB * D)[r] = make_float4(m, mv, sum, 0.0f);
          }
        }
        x += count;
        __syncwarp();
        if (lane == 0 && x < n_tiles) next_segment<OVER, SPLIT>(a, prefix, group, *cur);
        __syncwarp();
      }
    } else if (OVER == Over::ALL && threadIdx.x == 0) {
      const Cut none = {prefix[a.batch], 0, 0, 0, 0, 0, 0};
      a.cuts[cta] = none;
    }
    // blocks of rows that see nothing have no tiles: the CTAs share them out by heads
    for (int i = cta; OVER == Over::ALL && i < a.batch * c.n_heads; i += gridDim.x) {
      const int b = i / c.n_heads, head = i % c.n_heads;
      const Sequence sq = sequence_of<OVER>(a, b, nullptr);
      if (sq.n <= sq.len) continue;
      const Plan plan(sq, group);
      for (int block = 0; block < plan.blocks && plan.tiles(block) == 0; ++block) {
        const int rr = block * MB + (int)threadIdx.x;
        if (rr >= sq.n * group) continue;
        const int64_t row = sq.row0 + rr / group;
        const int qh = head * group + rr % group;
        char *out = static_cast<char *>(a.q.out) + 2 * (row * a.q.out_row_stride + qh * a.q.out_head_stride);
#pragma unroll 1
        for (int e = 0; e < D / 8; ++e) reinterpret_cast<uint4 *>(out)[e] = make_uint4(0u, 0u, 0u, 0u);
        if (a.q.d_lse) a.q.d_lse[row * a.q.q_heads + qh] = -INFINITY;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == ISSUE_WARP) tmem_free(tmem);
}

constexpr int JOIN_SHARE = 8, JOIN_THREADS = 128;  // CTAs to a cut segment's rows

// Joins the segment that CTA blockIdx.y's stretch begins in, if the one before holds its
// first part: what it needs of the plan the attending kernel has left beside the parts. At
// most one segment a CTA is cut, so only these are looked at, eight CTAs to one (2048 rows:
// 250 us for the call; 259 with four, 261 with a CTA to every 64 rows of every segment).
template <int D, int DT>
__global__ void __launch_bounds__(JOIN_THREADS, 8) kv_join_kernel(const __grid_constant__ AttentionArgs a) {
  const int c = blockIdx.y + 1, group = a.q.q_heads / a.c.n_heads;
  grid_dependency_wait();
  const Cut cut = a.cuts[c];
  if (cut.tile == 0) return;
  const Split split(a.cuts[0].total, a.ctas);
  const int64_t lo = split.start(c), begin = lo - cut.tile, end = begin + cut.tiles;
  const int64_t before = split.start(c - 1);
  if (before > begin) return;  // an earlier CTA begins in this segment too
  int last = c;
  while (last + 1 < split.ctas && split.start(last + 1) < end) ++last;
  const Sequence s = sequence_of(a, cut.b, nullptr);
  const int r0 = cut.block * MB, share = MB / JOIN_SHARE;
  const int from = blockIdx.x * share, to = min(from + share, s.n * group - r0);
  constexpr int64_t PART = (int64_t)MB * (D + 4);
  for (int u = from * (D / 4) + (int)threadIdx.x; u < to * (D / 4); u += JOIN_THREADS) {
    const int r = u / (D / 4), piece = u % (D / 4), rr = r0 + r;
    float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float top = NONE, topv = NONE, sum = 0.0f;
    for (int k = c - 1; k <= last; ++k) {  // in the order of the tokens
      const float *part = a.part + ((int64_t)k * 2 + (k < c && before < begin ? 1 : 0)) * PART;
      const float4 st = reinterpret_cast<const float4 *>(part + MB * D)[r];
      const float4 z = reinterpret_cast<const float4 *>(part)[r * (D / 4) + piece];
      const float m = fmaxf(top, st.x), mv = fmaxf(topv, st.y);
      const float keep = exp2_fast(topv - mv), f = exp2_fast(st.y - mv);
      sum = sum * exp2_fast(top - m) + st.z * exp2_fast(st.x - m);
      y = make_float4(y.x * keep + z.x * f, y.y * keep + z.y * f, y.z * keep + z.z * f,
                      y.w * keep + z.w * f);
      top = m;
      topv = mv;
    }
    const float f = sum > 0.0f ? exp2_fast(topv - top) / sum : 0.0f;
    const int64_t row = s.row0 + rr / group;
    const int qh = cut.head * group + rr % group;
    *reinterpret_cast<uint2 *>(static_cast<char *>(a.q.out) +
                               2 * (row * a.q.out_row_stride + qh * a.q.out_head_stride + 4 * piece)) =
        make_uint2(pack2<DT>(y.x * f, y.y * f), pack2<DT>(y.z * f, y.w * f));
    if (piece == 0 && a.q.d_lse)
      a.q.d_lse[row * a.q.q_heads + qh] = sum > 0.0f ? (top + log2f(sum)) * LN2 : -INFINITY;
  }
}

template <int D, int CODE, int DT, Over OVER, bool SPLIT>
int launch_for(AttentionArgs a, const DeviceInfo &dev, cudaStream_t s) {
  const auto kernel = kv_prefill_kernel<D, CODE, DT, OVER, SPLIT>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Memory<D>::bytes) !=
      cudaSuccess)
    return IBP_ERR_CUDA;
  // a warp that asks for more registers waits until others have given them up: they must
  // be there
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess ||
      16 * attr.numRegs < 8 * ROW_REGS + 4 * CONVERT_REGS + 4 * ISSUE_REGS)
    return IBP_ERR_CUDA;
  a.ctas = std::min(dev.sm_count, MAX_PREFILL_CTAS);
  if constexpr (OVER == Over::SHARED) {  // after the kernel that lays out the spans; joined by one of its own
    return launch_dependent(kernel, dim3((unsigned)a.ctas), dim3(THREADS), Memory<D>::bytes, s, a) == cudaSuccess
               ? IBP_OK
               : IBP_ERR_CUDA;
  } else {
    kernel<<<a.ctas, THREADS, Memory<D>::bytes, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return IBP_ERR_CUDA;
    if (a.ctas > 1 &&
        launch_dependent(kv_join_kernel<D, DT>, dim3(JOIN_SHARE, (unsigned)(a.ctas - 1)), dim3(JOIN_THREADS),
                         0, s, a) != cudaSuccess)
      return IBP_ERR_CUDA;
    return IBP_OK;
  }
}

template <int D, Over OVER, bool SPLIT>
int launch_types(const AttentionArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  if (a.c.code == IBP_KV_INT8)
    return a.q.dtype == IBP_BF16 ? launch_for<D, IBP_KV_INT8, IBP_BF16, OVER, SPLIT>(a, dev, s)
                                 : launch_for<D, IBP_KV_INT8, IBP_FP16, OVER, SPLIT>(a, dev, s);
  return a.q.dtype == IBP_BF16 ? launch_for<D, IBP_KV_E4M3, IBP_BF16, OVER, SPLIT>(a, dev, s)
                               : launch_for<D, IBP_KV_E4M3, IBP_FP16, OVER, SPLIT>(a, dev, s);
}

}  // namespace

size_t kv_prefill_scratch_bytes(const ibp_kv_cache &c) {
  return MAX_PREFILL_CTAS * (sizeof(Cut) + (size_t)2 * MB * (c.head_dim + 4) * sizeof(float));
}

int launch_kv_prefill(const ibp_kv_cache &c, const ibp_kv_query &q, void *d_scratch,
                      int32_t *d_status, cudaStream_t s) {
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  AttentionArgs a = {};
  a.c = c;
  a.q = q;
  a.status = d_status;
  a.wait_ns = gather_wait_limit_ns();
  a.withhold = withhold_plans();
  a.cuts = static_cast<Cut *>(d_scratch);
  a.part = reinterpret_cast<float *>(a.cuts + MAX_PREFILL_CTAS);
  for (a.b0 = 0; a.b0 < c.batch; a.b0 += BATCH) {
    a.batch = std::min(c.batch - a.b0, BATCH);
    if (int rc = c.head_dim == 64 ? launch_types<64, Over::ALL, false>(a, dev, s)
                                 : launch_types<128, Over::ALL, false>(a, dev, s))
      return rc;
  }
  return IBP_OK;
}

int launch_kv_prefill_shared(AttentionArgs a, bool split, cudaStream_t s) {
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  if (split)
    return a.c.head_dim == 64 ? launch_types<64, Over::SHARED, true>(a, dev, s)
                              : launch_types<128, Over::SHARED, true>(a, dev, s);
  return a.c.head_dim == 64 ? launch_types<64, Over::SHARED, false>(a, dev, s)
                            : launch_types<128, Over::SHARED, false>(a, dev, s);
}
PrefillShape prefill_shape(bool split) {
  DeviceInfo dev;
  return {split ? ROWS_OF<true> : ROWS_OF<false>, MB, TILE,
          device_info(&dev) == IBP_OK ? std::min(dev.sm_count, MAX_PREFILL_CTAS) : 0};
}

}  // namespace ibp
