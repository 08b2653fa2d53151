// Attention of a batch whose sequences share beginnings, over the 8-bit paged key/value cache
// (declared in include/ibp.h).
//
// A row's softmax over a shared beginning and over the rest of its sequence are joined by
// their sums of exponentials: with z_i = log2 of the i-th sum and o_i its normalised output,
//   z = log2(2^z_0 + 2^z_1),  out = o_0 2^(z_0 - z) + o_1 2^(z_1 - z).
// So a beginning is gone over once for the rows of all its sequences together, which fill the
// matrix unit, where each sequence by itself would read and convert it again.
//
// A small kernel lays out the spans; beginnings with more than 32 rows a K/V head go to the kernel
// for many rows, the rest of each sequence to the one for few, side by side on SMs that the
// layout shares out; a last kernel joins. (With fewer rows both go through the one for few
// together: two documents with 64 rows a head each take 92 us with the first way, 104 with the
// second.) 32 conversations behind 8,192 tokens, 32 query heads on 8 of 128: 48 us (undivided 89;
// floor 7); 16 answers to documents of 60,001 and 33,333, 32 on 4, e4m3: 75 us (undivided 107;
// floor 15). What bounds it: a tile takes the kernel for many rows 1.6 us for two halves whatever
// rows there are (fp16 of its codes made by four warps, shared memory that holds Q and both fp16
// tiles), 14 us go by before its first scores (layout 3.5, where its stretch begins 3, queries,
// pages, scales and codes one after another), and joining takes 4 us.
#include "ibp_kv_attend.cuh"

namespace ibp {

namespace {

constexpr int PLAN_THREADS = SHARE_SLAB;
constexpr int JOIN_WARPS = 4, JOIN_PARTS = 8;

// a / b of numbers that are not negative: a division in 64 bits takes several times as long
// as one in 32, which most of these fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

struct Side {
  int mb, part_rows, tile, ctas;  // rows of a segment and of a part, tokens of a tile, CTAs of the launch
  int cost;                       // of a tile: time that it takes an SM, in 0.1 us
  int split;                      // a part and a finished segment are in two results, mb rows apart
  const float *part;
};

struct ShareArgs {
  ibp_kv_cache c;
  ibp_kv_query q;
  int32_t *status;
  const int32_t *groups, *prefix;
  int n_groups, b0, batch;
  Side side[2];     // beginnings, the rest
  int together;     // both in one launch: tiles of the rest follow those of the beginnings
  int beginnings;   // spans kept for beginnings, the rest behind them
  Span *spans;      // [beginnings + batch]
  int64_t *total;   // [2] tiles of each side's launch
  int *active;      // [2] CTAs that share them
  const float *result, *result_lse2;  // as AttentionArgs::side
  int64_t side_rows;
};

// Exclusive sum over the block's threads; *all: the sum.
__device__ __forceinline__ int64_t sum_before(int64_t x, int64_t *warp_sum, int64_t *all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t run = x;
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(FULL, run, o);
    if (lane >= o) run += y;
  }
  __syncthreads();
  if (lane == 31) warp_sum[warp] = run;
  __syncthreads();
  int64_t before = 0, sum = 0;
  for (int k = 0; k < PLAN_THREADS / 32; ++k) {
    if (k < warp) before += warp_sum[k];
    sum += warp_sum[k];
  }
  *all = sum;
  return before + run - x;
}

// One CTA lays out the spans of up to SHARE_SLAB sequences (3.4 us: what it loads depends on one
// another, and it waits for its sums). A run of sequences of one group
// shares the whole pages of its prefix that none of its rows may not see; a run of one
// sequence shares nothing.
__global__ void __launch_bounds__(PLAN_THREADS) kv_share_plan_kernel(const __grid_constant__ ShareArgs a) {
  __shared__ int group_of[SHARE_SLAB], seen[SHARE_SLAB], members[SHARE_SLAB];
  __shared__ int first[SHARE_SLAB], last[SHARE_SLAB], place[SHARE_SLAB];
  __shared__ int64_t warp_sum[PLAN_THREADS / 32];
  const int t = threadIdx.x, b = a.b0 + t, heads = a.c.n_heads, group = a.q.q_heads / heads;
  const int P = a.c.page_tokens;
  const bool live = t < a.batch;
  grid_dependency_wait();  // for the kernel before it in the stream, which may have let it start
  grid_launch_dependents();
  // the last group that does not begin after the sequence, if it has it
  int mine = -1;
  if (live) {
    int lo = -1, hi = a.n_groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (__ldg(a.groups + mid) <= b) lo = mid; else hi = mid;
    }
    if (lo >= 0 && b < __ldg(a.groups + lo + 1)) mine = lo;
  }
  if (a.b0 == 0)
    for (int g = t; g < a.n_groups; g += PLAN_THREADS) {
      const int x = __ldg(a.groups + g), y = __ldg(a.groups + g + 1);
      if (x < 0 || y < x || y > a.c.batch) report(a.status, IBP_ERR_INDEX);
    }
  group_of[t] = mine;
  seen[t] = 0x7FFFFFFF;
  members[t] = last[t] = 0;
  first[t] = SHARE_SLAB - 1;
  __syncthreads();
  const bool starts = live && (t == 0 || mine < 0 || group_of[t - 1] != mine);
  int64_t runs;
  const int run = (int)sum_before(starts, warp_sum, &runs) + starts - 1;
  Span s = {};
  int n = 0, len = 0;
  int64_t lo = 0, hi = 0;
  if (live) {
    kv_row_range(a.q.d_cu, a.q.n_rows, a.q.max_q, b, a.status, &lo, &hi);
    if (hi - lo > a.q.max_q) report(a.status, IBP_ERR_INDEX);
    n = (int)min(hi - lo, a.q.max_q);
    len = kv_len(a.c, b, a.status);
    if (n > 0) {  // (one without rows may hold less than the others share)
      atomicMin(&first[run], t);
      atomicMax(&last[run], t);
      const int whole = mine >= 0 ? __ldg(a.prefix + mine) : 0;
      atomicMin(&seen[run], max(min(whole, len - n + 1), 0) / P * P);
      atomicAdd(&members[run], 1);
    }
  }
  __syncthreads();
  // beginnings: thread t lays out run t, those that are shared one after another
  bool shares = t < (int)runs && members[t] > 1 && seen[t] > 0;
  int64_t beginnings, total;
  const int at = (int)sum_before(shares, warp_sum, &beginnings);
  shares = shares && at < a.beginnings;  // (more of them: offsets that do not rise, recorded already)
  place[t] = shares ? at : -1;
  int64_t tiles = 0;
  __shared__ int segments;  // of the first beginning
  if (shares) {
    int64_t x, y, z, end;
    kv_row_range(a.q.d_cu, a.q.n_rows, a.q.max_q, a.b0 + first[t], nullptr, &x, &y);
    kv_row_range(a.q.d_cu, a.q.n_rows, a.q.max_q, a.b0 + last[t], nullptr, &z, &end);
    s.row0 = x;
    s.n = (int)max(min(end - x, (int64_t)0x3FFFFFFF), (int64_t)0);
    s.len = s.at = seen[t];
    s.table_at = (int64_t)(a.b0 + first[t]) * a.c.table_stride;
    const int64_t blocks = quotient((int64_t)s.n * group + a.side[0].mb - 1, a.side[0].mb);
    tiles = heads * blocks * ((s.len + a.side[0].tile - 1) / a.side[0].tile);
    if (at == 0) segments = (int)min(heads * blocks, (int64_t)0x3FFFFFFF);
  }
  s.before = sum_before(tiles, warp_sum, &total);
  if (shares) a.spans[at] = s;
  if (t >= (int)beginnings && t < a.beginnings) a.spans[t] = Span();
  const int64_t behind = a.together ? total : 0;
  if (t == 0) a.total[0] = total;
  __syncthreads();
  // the rest of each sequence
  s = Span();
  tiles = 0;
  if (live) {
    s.group = place[run];
    const int shared_tokens = s.group >= 0 ? seen[run] : 0;
    s.row0 = lo;
    s.n = n;
    s.len = len - shared_tokens;
    s.at = s.len - n;
    s.table_at = (int64_t)b * a.c.table_stride + shared_tokens / P;
    const int64_t blocks = quotient((int64_t)n * group + a.side[1].mb - 1, a.side[1].mb);
    tiles = heads * blocks * ((s.len + a.side[1].tile - 1) / a.side[1].tile);
  }
  s.before = behind + sum_before(tiles, warp_sum, &total);
  if (live) a.spans[a.beginnings + t] = s;
  if (t == 0) {
    a.total[1] = behind + total;
    if (a.together) {
      a.total[0] = behind + total;
      a.active[0] = a.active[1] = a.side[1].ctas;
    } else {
      // The two kernels run side by side: as many SMs to each as the tiles that it has take time
      // (32 conversations behind 8,192 tokens: 60 us one after the other).
      const int sms = a.side[0].ctas;
      const int64_t work = a.total[0] * a.side[0].cost, rest = total * a.side[1].cost;
      int mine = work == 0 ? 0 : rest == 0 ? sms : (int)min(max(sms * work / (work + rest), (int64_t)1), (int64_t)sms - 1);
      // no more than tiles; of one beginning, a whole number to each head and block of rows, so
      // that none goes over two (which takes it as long as four tiles more)
      mine = (int)min((int64_t)mine, a.total[0]);
      const int most = rest == 0 ? sms : sms - 1;
      if (beginnings == 1 && mine > segments) mine = min((mine + segments - 1) / segments, most / segments) * segments;
      a.active[0] = max(mine, 1);
      a.active[1] = max(a.side[1].ctas / sms * (sms - mine), 1);
    }
  }
}

__device__ __forceinline__ Span span_at(const Span *p) {
  static_assert(sizeof(Span) == 40, "five words of 64 bits");
  Span s;
  const long long *from = reinterpret_cast<const long long *>(p);
  long long w[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = __ldcg(from + i);
  s.row0 = w[0];
  s.table_at = w[1];
  s.before = w[2];
  s.n = (int)w[3];
  s.len = (int)(w[3] >> 32);
  s.at = (int)w[4];
  s.group = (int)(w[4] >> 32);
  return s;
}

// One row's result of one side: D/32 elements a lane, and log2 of its sum.
template <int D>
struct Half {
  static constexpr int V = D / 32;
  float y[V], z;
};

template <int V>
__device__ __forceinline__ void load_lane(const float *from, float *y) {
  if constexpr (V == 4) {
    const float4 v = __ldcg(reinterpret_cast<const float4 *>(from));
    y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
  } else {
    const float2 v = __ldcg(reinterpret_cast<const float2 *>(from));
    y[0] = v.x; y[1] = v.y;
  }
}

// Two results of one row over different tokens.
template <int D>
__device__ __forceinline__ Half<D> joined(const Half<D> &u, const Half<D> &v) {
  Half<D> h;
  const float top = fmaxf(u.z, v.z);
  const bool none = top == -INFINITY;  // neither has seen a token
  const float fu = none ? 0.0f : exp2_fast(u.z - top), fv = none ? 0.0f : exp2_fast(v.z - top);
  const float f = none ? 0.0f : 1.0f / (fu + fv);
#pragma unroll
  for (int e = 0; e < Half<D>::V; ++e) h.y[e] = (u.y[e] * fu + v.y[e] * fv) * f;
  h.z = none ? -INFINITY : top + log2f(fu + fv);
  return h;
}

// Where a row's results of one side lie (n 0: it has none). A segment that one CTA finished left
// its rows; the parts of the others are joined in their order, so that results do not depend on
// timing.
struct Where {
  int n, r;    // parts, two to a CTA if split; row in a part
  bool done;
  Parts p;
};
__device__ __forceinline__ Where where_of(const ShareArgs &a, int which, const Span &s, int64_t row, int qh) {
  Where w = {};
  // (rows outside the span: offsets that do not rise, recorded already)
  if (s.len <= 0 || row < s.row0 || row >= s.row0 + s.n) return w;
  const Side &side = a.side[which];
  const int group = a.q.q_heads / a.c.n_heads;
  const int64_t rr = (row - s.row0) * group + qh % group, block = quotient(rr, side.mb);
  const int64_t blocks = quotient((int64_t)s.n * group + side.mb - 1, side.mb);
  const int tiles = (s.len + side.tile - 1) / side.tile;
  w.r = (int)(rr - block * side.mb);
  // as parts_of, its divisions in 32 bits where they fit
  const int64_t total = __ldcg(a.total + which), start = s.before + (qh / group * blocks + block) * tiles;
  const int64_t ctas = min((int64_t)__ldcg(a.active + which), total);
  w.p.first = (int)quotient((start + 1) * ctas - 1, total);
  w.p.last = (int)quotient((start + tiles) * ctas - 1, total);
  w.p.second = quotient(total * w.p.first, ctas) < start;
  w.done = w.p.first == w.p.last;
  w.n = (w.done ? 1 : w.p.last - w.p.first + 1) << side.split;
  return w;
}

// One row's result over parts k0 .. k1 - 1.
template <int D>
__device__ __forceinline__ Half<D> half_of(const ShareArgs &a, int which, const Where &w, int k0, int k1,
                                           int64_t row, int qh) {
  constexpr int V = Half<D>::V;
  Half<D> h;
  for (int e = 0; e < V; ++e) h.y[e] = 0.0f;
  h.z = -INFINITY;
  if (k0 >= k1) return h;
  const Side &side = a.side[which];
  const int lane = threadIdx.x & 31;
  if (w.done) {
    for (int k = k0; k < k1; ++k) {
      const int64_t at = row * a.q.q_heads + qh + (which + 2 * k) * a.side_rows;
      Half<D> one;
      load_lane<V>(a.result + at * D + lane * V, one.y);
      one.z = __ldcg(a.result_lse2 + at);
      h = joined<D>(h, one);
    }
    return h;
  }
  const int64_t stride = (int64_t)side.part_rows * (D + 4);
  const int shift = side.split, n = k1;
  float top = NONE, topv = NONE, sum = 0.0f;
  for (; k0 < n; k0 += JOIN_PARTS) {
    float4 st[JOIN_PARTS];
    float y[JOIN_PARTS][V];
#pragma unroll
    for (int k = 0; k < JOIN_PARTS; ++k) {
      const int at = min(k0 + k, n - 1), cta = w.p.first + (at >> shift), rk = w.r + (shift ? at & 1 : 0) * side.mb;
      const float *part = side.part + ((int64_t)cta * 2 + (cta == w.p.first ? w.p.second : 0)) * stride;
      st[k] = __ldcg(reinterpret_cast<const float4 *>(part + side.part_rows * D) + rk);
      load_lane<V>(part + rk * D + lane * V, y[k]);
    }
    float m = top, mv = topv;
#pragma unroll
    for (int k = 0; k < JOIN_PARTS; ++k) {
      m = fmaxf(m, st[k].x);  // a part read twice does not raise it
      mv = fmaxf(mv, st[k].y);
    }
    const float fl = exp2_fast(top - m), fo = exp2_fast(topv - mv);
    sum *= fl;
#pragma unroll
    for (int e = 0; e < V; ++e) h.y[e] *= fo;
#pragma unroll
    for (int k = 0; k < JOIN_PARTS; ++k)
      if (k0 + k < n) {
        const float f = exp2_fast(st[k].y - mv);
        sum += st[k].z * exp2_fast(st[k].x - m);
#pragma unroll
        for (int e = 0; e < V; ++e) h.y[e] += y[k][e] * f;
      }
    top = m;
    topv = mv;
  }
  const float f = sum > 0.0f ? exp2_fast(topv - top) / sum : 0.0f;
#pragma unroll
  for (int e = 0; e < V; ++e) h.y[e] *= f;
  h.z = sum > 0.0f ? top + log2f(sum) : -INFINITY;
  return h;
}

// A warp to a row and query head, or (SHARE) a block of them: its warps share the parts of the
// beginning, of which a long one has dozens, the last takes the rest, and the first joins what
// they found.
template <int D, int DT, bool SHARE>
__global__ void __launch_bounds__(32 * JOIN_WARPS) kv_share_join_kernel(const __grid_constant__ ShareArgs a) {
  constexpr int V = Half<D>::V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t x = SHARE ? blockIdx.x : (int64_t)blockIdx.x * JOIN_WARPS + warp, each = a.q.max_q * a.q.q_heads;
  const int i = (int)quotient(x, each), in = (int)(x - i * each), j = in / a.q.q_heads, qh = in % a.q.q_heads;
  // The spans are there before the kernels that go over them let this one start (loads pass the
  // first-level cache), so that only their results are waited for.
  Span s = {}, from = {};
  if (i < a.batch) s = span_at(a.spans + a.beginnings + i);
  if (i < a.batch && s.group >= 0) from = span_at(a.spans + s.group);
  const int64_t row = s.row0 + j;
  const bool live = i < a.batch && j < s.n;
  Where first = {}, rest = {};
  if (live) {
    first = where_of(a, 0, from, row, qh);
    rest = where_of(a, 1, s, row, qh);
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (!live) return;
  Half<D> h;
  if constexpr (SHARE) {
    __shared__ float found[JOIN_WARPS][D], found_z[JOIN_WARPS];
    h = half_of<D>(a, 0, first, first.n * warp / JOIN_WARPS, first.n * (warp + 1) / JOIN_WARPS, row, qh);
    if (warp == JOIN_WARPS - 1) h = joined<D>(h, half_of<D>(a, 1, rest, 0, rest.n, row, qh));
    for (int e = 0; e < V; ++e) found[warp][lane * V + e] = h.y[e];
    if (lane == 0) found_z[warp] = h.z;
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int k = 1; k < JOIN_WARPS; ++k) {
      Half<D> other;
      for (int e = 0; e < V; ++e) other.y[e] = found[k][lane * V + e];
      other.z = found_z[k];
      h = joined<D>(h, other);
    }
  } else {
    h = joined<D>(half_of<D>(a, 0, first, 0, first.n, row, qh), half_of<D>(a, 1, rest, 0, rest.n, row, qh));
  }
  char *out = static_cast<char *>(a.q.out) +
              2 * (row * a.q.out_row_stride + qh * a.q.out_head_stride + lane * V);
  if constexpr (V == 4)
    *reinterpret_cast<uint2 *>(out) = make_uint2(pack2<DT>(h.y[0], h.y[1]), pack2<DT>(h.y[2], h.y[3]));
  else
    *reinterpret_cast<uint32_t *>(out) = pack2<DT>(h.y[0], h.y[1]);
  if (lane == 0 && a.q.d_lse) a.q.d_lse[row * a.q.q_heads + qh] = h.z * LN2;
}

// ---- host side

template <int D, int CODE, int DT>
int attend_rows(const AttentionArgs &a, int mb, const DeviceInfo &dev, cudaStream_t s) {
  switch (mb) {
    case 8: return launch_shape<D, CODE, DT, 1, 1, false, Over::SHARED>(a, dev, s);
    case 16: return launch_shape<D, CODE, DT, 2, 1, false, Over::SHARED>(a, dev, s);
    case 32: return launch_shape<D, CODE, DT, 2, 2, false, Over::SHARED>(a, dev, s);
    default: return launch_shape<D, CODE, DT, 2, 4, false, Over::SHARED>(a, dev, s);
  }
}
template <int D>
int attend_types(const AttentionArgs &a, int mb, const DeviceInfo &dev, cudaStream_t s) {
  if (a.c.code == IBP_KV_INT8)
    return a.q.dtype == IBP_BF16 ? attend_rows<D, IBP_KV_INT8, IBP_BF16>(a, mb, dev, s)
                                 : attend_rows<D, IBP_KV_INT8, IBP_FP16>(a, mb, dev, s);
  return a.q.dtype == IBP_BF16 ? attend_rows<D, IBP_KV_E4M3, IBP_BF16>(a, mb, dev, s)
                               : attend_rows<D, IBP_KV_E4M3, IBP_FP16>(a, mb, dev, s);
}

template <int D>
int launch_join(const ShareArgs &a, bool share, int64_t blocks, cudaStream_t s) {
  const bool bf16 = a.q.dtype == IBP_BF16;
  const auto join = share ? (bf16 ? kv_share_join_kernel<D, IBP_BF16, true> : kv_share_join_kernel<D, IBP_FP16, true>)
                          : (bf16 ? kv_share_join_kernel<D, IBP_BF16, false> : kv_share_join_kernel<D, IBP_FP16, false>);
  return launch_dependent(join, dim3((unsigned)blocks), dim3(32 * JOIN_WARPS), 0, s, a) == cudaSuccess ? IBP_OK : IBP_ERR_CUDA;
}

// CTAs of the kernel for few rows in segments of mb.
int attend_ctas(int mb, const DeviceInfo &dev) { return std::min((mb == 8 ? 3 : 2) * dev.sm_count, MAX_CTAS); }

constexpr int64_t ALONE_BYTES = int64_t(64) << 20;

// How a call is divided: rows of a segment, and whether beginnings go to the kernel for many
// rows or along with the rest. alone: not divided at all.
struct Division {
  bool alone, many, split;
  int mb;
};
Division division_of(const ibp_kv_cache &c, int64_t n_rows, int64_t max_q, int q_heads, int64_t n_groups,
                     int64_t group_rows) {
  const int64_t group = q_heads / c.n_heads, each = std::min(max_q, n_rows) * group;
  const int64_t all = std::max(std::min(group_rows, n_rows) * group, each);
  Division d;
  // Not divided: many rows of every sequence, which arithmetic bounds; and where all that the
  // tables can hold is read within the time that laying out, a second kernel and joining take
  // (4 sequences of 777 to 877 tokens, 8 heads of 128, tables of 7 MB: 12 us, 18 divided; 40 of up
  // to 5,004, 4 heads of 64, 104 MB: 49 us, 41 divided). It goes by what the tables can hold, as
  // the lengths are on the device: through tables that are wide for what is held little is
  // divided too and takes the longer way (those 4 behind tables for 65,536 tokens 18.6 us, 32
  // conversations behind 777 tokens 29 where 21 undivided; 8 behind 8,192 36 and 31; behind 60,001
  // 86 and 145).
  const int64_t held = (int64_t)c.batch * c.table_cols * c.page_tokens * c.n_heads * 2 * c.head_dim;
  d.alone = each > 64 || n_groups == 0 || held <= ALONE_BYTES;
  d.many = all > 32;
  d.split = all <= prefill_shape(true).rows;
  d.mb = rows_of(d.many ? each : all);
  return d;
}

struct ShareLayout {
  size_t spans, parts[2], result, lse2, bytes;
};
ShareLayout share_layout(const ibp_kv_cache &c, const Division &d, int64_t n_rows, int q_heads) {
  const size_t row = (c.head_dim + 4) * sizeof(float), rows = (size_t)n_rows * q_heads;
  ShareLayout y;
  y.spans = 0;
  y.parts[1] = (2 * SHARE_SLAB * sizeof(Span) + 2 * sizeof(int64_t) + 2 * sizeof(int) + 255) / 256 * 256;
  y.parts[0] = y.parts[1] + (size_t)MAX_CTAS * 2 * d.mb * row;
  y.result = y.parts[0] + (d.many ? (size_t)MAX_PREFILL_CTAS * 2 * prefill_shape(d.split).part_rows * row : 0);
  y.lse2 = y.result + 3 * rows * c.head_dim * sizeof(float);
  y.bytes = y.lse2 + (3 * rows * sizeof(float) + 255) / 256 * 256;
  return y;
}

}  // namespace

size_t kv_shared_scratch_bytes(const ibp_kv_cache &c, int64_t n_rows, int64_t max_q, int q_heads,
                               int64_t n_groups, int64_t group_rows) {
  const Division d = division_of(c, n_rows, max_q, q_heads, n_groups, group_rows);
  if (d.alone) return kv_attention_scratch_bytes(c, n_rows, max_q, q_heads, false);
  return share_layout(c, d, n_rows, q_heads).bytes;
}

int launch_kv_attention_shared(const ibp_kv_cache &c, const ibp_kv_query &query, const int32_t *d_groups,
                               const int32_t *d_prefix, int64_t n_groups, int64_t group_rows, void *d_scratch,
                               int32_t *d_status, cudaStream_t s) {
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  const Division d = division_of(c, query.n_rows, query.max_q, query.q_heads, n_groups, group_rows);
  if (d.alone) return launch_kv_attention(c, query, d_scratch, d_status, s);
  const ShareLayout y = share_layout(c, d, query.n_rows, query.q_heads);
  char *base = static_cast<char *>(d_scratch);
  ShareArgs a = {};
  a.c = c;
  a.q = query;
  a.q.max_q = std::min(query.max_q, query.n_rows);
  a.status = d_status;
  a.groups = d_groups;
  a.prefix = d_prefix;
  a.n_groups = (int)n_groups;
  a.together = !d.many;
  a.spans = reinterpret_cast<Span *>(base + y.spans);
  a.total = reinterpret_cast<int64_t *>(a.spans + 2 * SHARE_SLAB);
  a.active = reinterpret_cast<int *>(a.total + 2);
  a.result = reinterpret_cast<float *>(base + y.result);
  a.result_lse2 = reinterpret_cast<float *>(base + y.lse2);
  a.side_rows = query.n_rows * query.q_heads;
  // (costs: what tiles of long sequences took when kernels had the GPU to themselves)
  a.side[1] = {d.mb, d.mb, TILE, attend_ctas(d.mb, dev), d.mb <= 16 ? 5 : d.mb == 32 ? 9 : 18, 0, reinterpret_cast<float *>(base + y.parts[1])};
  a.side[0] = a.side[1];
  const PrefillShape many = prefill_shape(d.split);
  if (d.many)
    a.side[0] = {many.rows, many.part_rows, many.tile, many.ctas, d.split ? 24 : 36, d.split, reinterpret_cast<float *>(base + y.parts[0])};

  AttentionArgs t = {};
  t.c = c;
  t.q = a.q;
  t.status = d_status;
  t.wait_ns = gather_wait_limit_ns();
  t.withhold = withhold_plans();
  t.spans = a.spans;
  t.side = const_cast<float *>(a.result);
  t.side_lse2 = const_cast<float *>(a.result_lse2);
  t.side_rows = a.side_rows;
  for (a.b0 = 0; a.b0 < c.batch; a.b0 += SHARE_SLAB) {
    a.batch = std::min(c.batch - a.b0, SHARE_SLAB);
    // of a slab's sequences, two at least have each shared beginning
    a.beginnings = t.beginnings = (int)std::min<int64_t>(n_groups, (a.batch + 1) / 2);
    if (launch_dependent(kv_share_plan_kernel, dim3(1), dim3(PLAN_THREADS), 0, s, a) != cudaSuccess) return IBP_ERR_CUDA;
    if (d.many) {
      t.b0 = 0;
      t.batch = a.beginnings;
      t.part = const_cast<float *>(a.side[0].part);
      t.active = a.active;
      t.beside = 0;
      if (int rc = launch_kv_prefill_shared(t, d.split, s)) return rc;
    }
    t.b0 = d.many ? a.beginnings : 0;
    t.batch = a.beginnings + a.batch - t.b0;
    t.part = const_cast<float *>(a.side[1].part);
    t.active = a.active + 1;
    t.beside = d.many;
    if (int rc = c.head_dim == 64 ? attend_types<64>(t, d.mb, dev, s) : attend_types<128>(t, d.mb, dev, s)) return rc;
    // Several warps to a row while all rows are there at once (512 rows with 50 parts: 9 us, 4 with
    // four warps to each; 4,480 with two: 5 and 11).
    const int64_t rows = a.batch * a.q.max_q * query.q_heads;
    const bool share = rows <= 4 * (int64_t)dev.sm_count;
    const int64_t blocks = share ? rows : (rows + JOIN_WARPS - 1) / JOIN_WARPS;
    if (blocks > 0x7FFFFFFF) return IBP_ERR_UNSUPPORTED;
    if (int rc = c.head_dim == 64 ? launch_join<64>(a, share, blocks, s) : launch_join<128>(a, share, blocks, s)) return rc;
  }
  return IBP_OK;
}

}  // namespace ibp
