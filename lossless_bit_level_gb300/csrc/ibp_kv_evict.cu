// Eviction from the 8-bit paged key/value cache by accumulated attention weight
// (declared in include/ibp.h): which tokens stay, then their values requantised into
// the destination's pages.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "ibp_kv_device.cuh"

namespace cg = cooperative_groups;

namespace ibp {

namespace {

// The kept set of one (sequence, head): the need-th largest of the weights that compete,
// found from the top bits down in three passes that count the keys by 11, 11 and 10 of
// their bits, then one pass that counts and one that lists, in token order, the keys
// above it and the first of those equal to it. A cluster of CTAs shares one long
// sequence: each counts its own stretch, adds up an equal share of the bins over all CTAs
// through distributed shared memory and hands the sums to the others, and every CTA finds
// the same threshold. The weights are read from memory once and the passes go over the
// keys in shared memory; what bounds it is the passes one after another, with a barrier
// and a scan of the bins between them, not the bytes: 256 lists of up to 4,096 weights take
// 17 us, 16 lists of 61,000 to 100,003 (six times as much for a CTA) 40 us in clusters.
constexpr int SELECT_THREADS[2] = {512, 1024};  // of a lone CTA (four fit an SM), of one in a cluster
constexpr int BINS = 2048;
constexpr int MAX_CLUSTER = 8;
constexpr int MAX_CACHED = 24576;  // keys of a CTA's stretch kept in shared memory (96 KB)

// Unsigned order of the weights: a larger key is a larger weight, NaN lowest, -0 = 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.0f ? 0.0f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct SelectArgs {
  ibp_kv_cache c;
  const float *weights;
  int64_t stride, new_stride;
  int budget, recent, cached;  // cached: keys that the shared memory given holds
  int most;                    // tokens that can be kept: the smaller of budget and capacity
  int page_shift;
  int32_t *new_lens;
  float *new_weights;
  int32_t *kept;
  int64_t *list;  // [batch][n_heads][most]: page * page_tokens + slot, or -1
  int32_t *status;
};

template <bool CLUSTER>
__global__ void __launch_bounds__(SELECT_THREADS[CLUSTER], CLUSTER ? 1 : 4)
    kv_select_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int THREADS = SELECT_THREADS[CLUSTER], WARPS = THREADS / 32;
  extern __shared__ uint32_t cache[];
  __shared__ uint32_t hist[BINS], sums[CLUSTER ? BINS : 1];
  __shared__ int32_t pages[MAX_CACHED / 16 + 2];  // of the cached stretch
  __shared__ uint32_t warp_sum[WARPS];
  __shared__ uint32_t found[2];             // bin, what is still needed within it
  __shared__ uint2 warp_count[WARPS];  // keys above and equal, of each warp's stretch
  __shared__ uint2 cta_count;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = CLUSTER ? (int)cluster.num_blocks() : 1, rank = CLUSTER ? (int)cluster.block_rank() : 0;
  const ibp_kv_cache &c = a.c;
  const int64_t bh = blockIdx.x / C;
  const int b = (int)(bh / c.n_heads), head = (int)(bh % c.n_heads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  grid_launch_dependents();
  const float *w = a.weights + bh * a.stride;
  const int len = kv_len(c, b, a.status), out = min(len, a.budget);
  int64_t *row = a.list + bh * a.most;
  int32_t *kept = a.kept ? a.kept + bh * a.budget : nullptr;
  float *new_w = a.new_weights ? a.new_weights + bh * a.new_stride : nullptr;
  auto put = [&](int at, int t, float x, int page) {
    row[at] = page < 0 ? -1 : ((int64_t)page << a.page_shift) + (t & (c.page_tokens - 1));
    if (kept) kept[at] = t;
    if (new_w) new_w[at] = x;
  };
  const int all_threads = C * THREADS, all_tid = rank * THREADS + tid;

  for (int64_t i = out + all_tid; i < a.budget; i += all_threads)
    if (kept) kept[i] = -1;
  if (new_w)
    for (int64_t i = out + all_tid; i < a.new_stride; i += all_threads) new_w[i] = 0.0f;
  if (head == 0 && all_tid == 0) a.new_lens[b] = out;
  // tokens kept without a contest: all of a short sequence, else the last `recent`
  const bool all = len <= a.budget;
  const int open = all ? 0 : len - a.recent, room = all ? 0 : a.budget - a.recent;
  for (int t = open + all_tid; t < len; t += all_threads)
    put(room + t - open, t, new_w ? w[t] : 0.0f, kv_page(c, b, t >> a.page_shift, a.status));
  if (room == 0) return;  // the same for every CTA of the cluster

  // this CTA's stretch of the competing tokens, in whole 32-token pieces a warp
  const int per_warp = ((open + C * THREADS - 1) / (C * THREADS)) * 32;
  const int64_t first64 = (int64_t)(rank * WARPS + warp) * per_warp;
  const int first = (int)min(first64, (int64_t)open);
  const int last = (int)min(first64 + per_warp, (int64_t)open);

  // the stretch is gone over five times: as keys in shared memory, where they fit
  const int64_t cta_first = (int64_t)rank * WARPS * per_warp;
  const bool in_cache = WARPS * per_warp <= a.cached;
  const int first_page = (int)(min(cta_first, (int64_t)open) >> a.page_shift);
  if (in_cache) {
    const int n = (int)max(min((int64_t)open - cta_first, (int64_t)WARPS * per_warp), (int64_t)0);
#pragma unroll 8
    for (int i = tid; i < n; i += THREADS) cache[i] = weight_key(__ldg(w + cta_first + i));
    if (n > 0)
      for (int i = first_page + tid; i <= (int)((cta_first + n - 1) >> a.page_shift); i += THREADS)
        pages[i - first_page] = __ldg(c.d_table + (int64_t)b * c.table_stride + i);
  }
  auto key_at = [&](int t) {
    return in_cache ? cache[t - (int)cta_first] : weight_key(__ldg(w + t));
  };

  uint32_t need = (uint32_t)room, prefix = 0;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
    const uint32_t above = pass == 0 ? 0u : FULL << (pass == 1 ? 21 : 10);
    for (int i = tid; i < bins; i += THREADS) hist[i] = 0;
    __syncthreads();
    for (int t0 = first; t0 < last; t0 += 128) {
      uint32_t key[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + e * 32 + lane;
        key[e] = t < last ? key_at(t) : 0u;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = t0 + e * 32 + lane < last && ((key[e] ^ prefix) & above) == 0;
        if (in) atomicAdd(&hist[(key[e] >> shift) & (bins - 1)], 1u);
      }
    }
    __syncthreads();
    const uint32_t *count = hist;
    if constexpr (CLUSTER) {
      cluster.sync();
      const int share = bins / C;
      for (int i = rank * share + tid; i < (rank + 1) * share; i += THREADS) {
        uint32_t n = 0;
#pragma unroll
        for (int k = 0; k < MAX_CLUSTER; ++k)
          if (k < C) n += cluster.map_shared_rank(hist, k)[i];
#pragma unroll
        for (int k = 0; k < MAX_CLUSTER; ++k)
          if (k < C) cluster.map_shared_rank(sums, k)[i] = n;
      }
      cluster.sync();
      count = sums;
    }
    // bins from the top: thread i holds a few of them, highest first
    constexpr int most = BINS / THREADS;
    const int per = bins / THREADS;
    uint32_t n[most] = {};
#pragma unroll
    for (int e = 0; e < most; ++e)
      if (e < per) n[e] = count[bins - 1 - (tid * per + e)];
    uint32_t sum = 0;
#pragma unroll
    for (int e = 0; e < most; ++e) sum += n[e];
    uint32_t run = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(FULL, run, o);
      if (lane >= o) run += y;
    }
    if (lane == 31) warp_sum[warp] = run;
    __syncthreads();
    if (warp == 0) {
      uint32_t y = lane < WARPS ? warp_sum[lane] : 0u, z = y;
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(FULL, z, o);
        if (lane >= o) z += u;
      }
      if (lane < WARPS) warp_sum[lane] = z - y;
    }
    __syncthreads();
    uint32_t before = warp_sum[warp] + run - sum;  // keys in higher bins
#pragma unroll
    for (int e = 0; e < most; ++e) {
      if (e < per && before < need && before + n[e] >= need) {
        found[0] = (uint32_t)(bins - 1 - (tid * per + e));
        found[1] = need - before;
      }
      before += n[e];
    }
    __syncthreads();
    prefix |= found[0] << shift;
    need = found[1];
  }

  // keys above the threshold, and equal to it, in each stretch
  uint32_t gt = 0, eq = 0;
  for (int t0 = first; t0 < last; t0 += 32) {
    const bool in = t0 + lane < last;
    const uint32_t key = in ? key_at(t0 + lane) : 0u;
    gt += __popc(__ballot_sync(FULL, in && key > prefix));
    eq += __popc(__ballot_sync(FULL, in && key == prefix));
  }
  if (lane == 0) warp_count[warp] = make_uint2(gt, eq);
  __syncthreads();
  if (tid == 0) {
    uint2 s = make_uint2(0, 0);
    for (int k = 0; k < WARPS; ++k) {
      s.x += warp_count[k].x;
      s.y += warp_count[k].y;
    }
    cta_count = s;
  }
  if constexpr (CLUSTER) cluster.sync();
  uint32_t gt_before = 0, eq_before = 0;
  for (int k = 0; k < rank; ++k) {
    const uint2 s = *cluster.map_shared_rank(&cta_count, k);
    gt_before += s.x;
    eq_before += s.y;
  }
  for (int k = 0; k < warp; ++k) {
    gt_before += warp_count[k].x;
    eq_before += warp_count[k].y;
  }
  const uint32_t lower = (1u << lane) - 1u;
  for (int t0 = first; t0 < last; t0 += 32) {
    const int t = t0 + lane;
    const bool in = t < last;
    const uint32_t key = in ? key_at(t) : 0u;
    const unsigned g = __ballot_sync(FULL, in && key > prefix);
    const unsigned e = __ballot_sync(FULL, in && key == prefix);
    const uint32_t mine_g = gt_before + __popc(g & lower), mine_e = eq_before + __popc(e & lower);
    if (in && (key > prefix || (key == prefix && mine_e < need))) {
      const uint32_t at = mine_g + min(mine_e, need);
      if (at < (uint32_t)room) {
        const int col = t >> a.page_shift;
        int page = in_cache ? pages[col - first_page] : kv_page(c, b, col, a.status);
        if (page < 0 || page >= c.n_pages) {
          report(a.status, IBP_ERR_INDEX);
          page = -1;
        }
        put((int)at, t, new_w ? __ldg(w + t) : 0.0f, page);
      }
    }
    gt_before += __popc(g);
    eq_before += __popc(e);
  }
  if constexpr (CLUSTER) cluster.sync();  // no CTA leaves while another reads its counts
}

// Largest magnitude among 16 codes. Bytes are compared as the upper halves of 16-bit
// lanes: what lies below them cannot change which upper byte is the largest.
template <int CODE>
__device__ __forceinline__ float largest_code(uint4 w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  if constexpr (CODE == IBP_KV_INT8) {
    uint32_t hi = 0u, lo = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hi = max_s16x2(max_s16x2(hi, u[i]), u[i] << 8);
      lo = min_s16x2(min_s16x2(lo, u[i]), u[i] << 8);
    }
    const int top = max((int)hi >> 24, (int)(hi << 16) >> 24);
    const int low = min((int)lo >> 24, (int)(lo << 16) >> 24);
    return (float)max(top, -low);
  } else {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = max_u16x2(max_u16x2(m, u[i] & 0x7F7F7F7Fu), (u[i] << 8) & 0x7F007F00u);
    float x[4];
    kv_decode4<CODE>(max(m >> 24, (m >> 8) & 0xFFu), x);
    return x[0];
  }
}

// The larger of two numbers, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// The largest finite magnitude of a token's 16 values, one by one.
template <int CODE>
__device__ __noinline__ float largest_finite(uint4 w, float scale) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  float most = 0.0f;
  for (int i = 0; i < 4; ++i) {
    float x[4];
    kv_decode4<CODE>(u[i], x);
    for (int k = 0; k < 4; ++k) most = fmaxf(most, finite_abs(__fmul_rn(x[k], scale)));
  }
  return most;
}

// One CTA per (sequence, head, destination page, K or V): the kept tokens' values,
// their maximum, their codes. A token's codes share one scale, so its largest value is
// its largest code times that scale (rounding keeps the order): the maximum is taken over
// codes, and the values are formed once. (A product that is not finite comes from a NaN code or
// from a scale that no append writes, in a pool that a caller filled: the thread's values are
// then gone over one by one.) The scattered rows are read once and stay in
// registers; a row of a head is whole 32-byte sectors (64 or 128 bytes), so scattering costs
// little, and what bounds it is instruction issue (64 % of the slots at 8 sequences cut
// from at most 4,096 to 2,048 tokens, 32 heads of 128: 52 us, 5.2 TB/s) beside the wait for
// list entries and then for rows. At most 80 registers, so that an SM holds 704 threads.
template <int P, int D, int CODE>
__global__ void __launch_bounds__(Tile<P, D>::threads, 704 / Tile<P, D>::threads)
    kv_move_kernel(ibp_kv_cache c, ibp_kv_cache dst, int most, const int64_t *list,
                   int32_t *status) {
  constexpr int T = Tile<P, D>::threads, G = Tile<P, D>::per_thread, GD = D / 16,
                STEP = Tile<P, D>::step;
  __shared__ uint32_t sm[32];
  const int head = blockIdx.y % c.n_heads;
  const bool is_v = (int)blockIdx.y >= c.n_heads;
  const int b = blockIdx.z, t0 = blockIdx.x * P + threadIdx.x / GD;
  const int out = min(kv_len(c, b, nullptr), most);
  const int to = (int)blockIdx.x * P < out ? kv_page(dst, b, blockIdx.x, status) : -1;
  const int64_t *row = list + ((int64_t)b * c.n_heads + head) * most + t0;
  const char *codes = static_cast<const char *>(is_v ? c.v_codes : c.k_codes) + (threadIdx.x % GD) * 16;
  const float *scales = is_v ? c.v_scales : c.k_scales;
  grid_dependency_wait();  // for the list; also before a return: what comes next may be
  if (to < 0) return;      // ordered behind this grid alone
  int64_t from[G];
#pragma unroll
  for (int g = 0; g < G; ++g) from[g] = t0 + g * STEP < out ? row[g * STEP] : -1;
  uint4 w[G];
  float scale[G], largest = 0.0f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    w[g] = make_uint4(0u, 0u, 0u, 0u);
    scale[g] = 0.0f;
    if (from[g] >= 0) {
      const int64_t tile = from[g] / P * c.n_heads + head;
      scale[g] = __ldg(scales + tile);
      w[g] = __ldg(reinterpret_cast<const uint4 *>(codes + (tile * P + from[g] % P) * D));
    }
  }
#pragma unroll
  for (int g = 0; g < G; ++g)
    largest = max_nan(largest, __fmul_rn(largest_code<CODE>(w[g]), fabsf(scale[g])));
  const bool odd = !(largest <= FLT_MAX);
  if (odd) {
    largest = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) largest = fmaxf(largest, largest_finite<CODE>(w[g], scale[g]));
  }
  largest = __uint_as_float(block_max(__float_as_uint(largest), sm));
  const float new_scale = kv_scale<CODE>(largest), inverse = kv_inverse(new_scale);
  if (threadIdx.x == 0)
    (is_v ? dst.v_scales : dst.k_scales)[(int64_t)to * c.n_heads + head] = new_scale;
  uint4 *put = reinterpret_cast<uint4 *>(static_cast<char *>(is_v ? dst.v_codes : dst.k_codes) +
                                         kv_tile(dst, to, head)) + threadIdx.x;
  auto put_all = [&](auto saturate) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t u[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[4];
        kv_decode4<CODE>(u[i], x);
        mul4(x, scale[g]);
        mul4(x, inverse);
        v[i] = decltype(saturate)::value ? kv_encode4_any<CODE>(x[0], x[1], x[2], x[3])
                                         : kv_encode4<CODE>(x[0], x[1], x[2], x[3]);
      }
      if (t0 + g * STEP < out) put[g * T] = make_uint4(v[0], v[1], v[2], v[3]);
    }
  };
  if (new_scale < 0x1p120f && !odd)
    put_all(std::false_type());
  else
    put_all(std::true_type());
}

template <int P, int D>
int move_code(const ibp_kv_cache &c, const ibp_kv_cache &dst, int most, const int64_t *list,
              int32_t *status, cudaStream_t s) {
  const dim3 grid((unsigned)((most + P - 1) / P), (unsigned)(2 * c.n_heads), (unsigned)c.batch);
  if (grid.x == 0) return IBP_OK;
  const auto kernel = c.code == IBP_KV_INT8 ? kv_move_kernel<P, D, IBP_KV_INT8>
                                            : kv_move_kernel<P, D, IBP_KV_E4M3>;
  return launch_dependent(kernel, grid, dim3(Tile<P, D>::threads), 0, s, c, dst, most, list,
                          status) == cudaSuccess
             ? IBP_OK
             : IBP_ERR_CUDA;
}

template <int P>
int move_dim(const ibp_kv_cache &c, const ibp_kv_cache &dst, int most, const int64_t *list,
             int32_t *status, cudaStream_t s) {
  return c.head_dim == 64 ? move_code<P, 64>(c, dst, most, list, status, s)
                          : move_code<P, 128>(c, dst, most, list, status, s);
}

}  // namespace

// Tokens of a list that can be kept.
static int most_of(const ibp_kv_cache &c, int64_t budget) {
  return (int)std::min(budget, (int64_t)c.table_cols * c.page_tokens);
}

size_t kv_evict_scratch_bytes(const ibp_kv_cache &c, int64_t budget) {
  const size_t bytes = (size_t)c.batch * c.n_heads * most_of(c, budget) * sizeof(int64_t);
  return std::max<size_t>((bytes + 15) / 16 * 16, 16);
}

int launch_kv_evict(const ibp_kv_cache &c, const float *d_weights, int64_t weights_stride,
                    int64_t budget, int64_t recent, const ibp_kv_cache &dst, int32_t *d_new_lens,
                    float *d_new_weights, int64_t new_weights_stride, int32_t *d_kept,
                    void *d_scratch, int32_t *d_status, cudaStream_t s) {
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  int64_t *list = static_cast<int64_t *>(d_scratch);
  // More CTAs a list while there are SMs for them and 4096 tokens for each. Whole calls with
  // clusters | without: 8 lists of 4,096 tokens (two CTAs would have 2048 each) 19 us either
  // way, of 8,192 25 | 27 us, of 16,384 27 | 40, of 65,536 43 | 236; 64 lists of 16,384
  // 56 | 64, of 65,536 191 | 335 (a lone CTA cannot keep that many keys).
  const int64_t cap = (int64_t)c.table_cols * c.page_tokens, rows = (int64_t)c.batch * c.n_heads;
  int cluster = 1;
  while (cluster < MAX_CLUSTER && rows * cluster * 2 <= dev.sm_count &&
         cap >= (int64_t)cluster * 2 * 4096)
    cluster *= 2;
  const int threads = SELECT_THREADS[cluster > 1];
  const int most = most_of(c, budget);
  const int64_t stretch = (cap + cluster * threads - 1) / (cluster * threads) * threads;
  const int cached = stretch <= MAX_CACHED ? (int)stretch : 0;
  const SelectArgs a = {c,           d_weights,   weights_stride, new_weights_stride,
                        (int)budget, (int)recent, cached, most,
                        __builtin_ctz((unsigned)c.page_tokens), d_new_lens,
                        d_new_weights, d_kept, list, d_status};
  const auto select = cluster > 1 ? kv_select_kernel<true> : kv_select_kernel<false>;
  if (cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           MAX_CACHED * (int)sizeof(uint32_t)) != cudaSuccess)
    return IBP_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = (size_t)cached * sizeof(uint32_t);
  cfg.gridDim = dim3((unsigned)(rows * cluster));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, select, a) != cudaSuccess) return IBP_ERR_CUDA;
  switch (c.page_tokens) {
    case 16: return move_dim<16>(c, dst, most, list, d_status, s);
    case 32: return move_dim<32>(c, dst, most, list, d_status, s);
    case 64: return move_dim<64>(c, dst, most, list, d_status, s);
    default: return move_dim<128>(c, dst, most, list, d_status, s);
  }
}

}  // namespace ibp
