// Attention over the 8-bit paged key/value cache (declared in include/ibp.h; the formulas
// stand at the head of ibp_kv_attend.cuh).
#include <algorithm>
#include <numeric>

#include "ibp_kv_attend.cuh"

namespace ibp {

namespace {

// ---- host side -------------------------------------------------------------------

int score_cols_of(const ibp_kv_cache &c) {
  return (c.table_cols * c.page_tokens + TILE - 1) / TILE * TILE;
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

template <int D, int CODE, int DT>
int launch_rows(const AttentionArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  const bool w = a.q.d_weights != nullptr;
  switch (rows_of(launch_rows_of(a) * (a.q.q_heads / a.c.n_heads))) {
    case 8:
      return w ? launch_shape<D, CODE, DT, 1, 1, true, Over::ALL>(a, dev, s)
               : launch_shape<D, CODE, DT, 1, 1, false, Over::ALL>(a, dev, s);
    case 16:
      return w ? launch_shape<D, CODE, DT, 2, 1, true, Over::ALL>(a, dev, s)
               : launch_shape<D, CODE, DT, 2, 1, false, Over::ALL>(a, dev, s);
    case 32:
      return w ? launch_shape<D, CODE, DT, 2, 2, true, Over::ALL>(a, dev, s)
               : launch_shape<D, CODE, DT, 2, 2, false, Over::ALL>(a, dev, s);
    default: return launch_shape<D, CODE, DT, 2, 4, true, Over::ALL>(a, dev, s);  // weights: see many_rows
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
  AttentionArgs a = {};
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
