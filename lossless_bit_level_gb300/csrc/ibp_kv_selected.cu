// Attention over the selected pages of the 8-bit paged key/value cache (declared in
// include/ibp.h): the kernel for few query rows over the pages that a list names. A list is gone
// over as if it were a sequence; all that differs is where a tile's pages come from (two look-ups
// more, a batch of pages ahead of the copies). 16 sequences, 8 heads of 128, 64 pages of 32 tokens
// each (67 MB of codes): 20 us, 3.4 TB/s, of which 5 go by before the first tile; the same
// sequences whole (35,000 to 60,001 tokens) take 246.
#include "ibp_kv_attend.cuh"

namespace ibp {

namespace {

template <int D, int CODE, int DT>
int launch_rows(const AttentionArgs &a, const DeviceInfo &dev, cudaStream_t s) {
  switch (rows_of(a.q.max_q * (a.q.q_heads / a.c.n_heads))) {
    case 8: return launch_shape<D, CODE, DT, 1, 1, false, Over::SELECTED>(a, dev, s);
    case 16: return launch_shape<D, CODE, DT, 2, 1, false, Over::SELECTED>(a, dev, s);
    default: return launch_shape<D, CODE, DT, 2, 2, false, Over::SELECTED>(a, dev, s);
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

// More than 32 rows are gone over in segments of 32.
size_t kv_selected_scratch_bytes(const ibp_kv_cache &c, int64_t n_rows, int64_t max_q, int q_heads) {
  const int mb = std::min(rows_of(std::min(max_q, n_rows) * (q_heads / c.n_heads)), 32);
  return (size_t)MAX_CTAS * 2 * mb * (c.head_dim + 4) * sizeof(float);
}

int launch_kv_attention_selected(const ibp_kv_cache &c, const ibp_kv_query &query, const int32_t *d_columns,
                                 int64_t pages, void *d_scratch, int32_t *d_status, cudaStream_t s) {
  DeviceInfo dev;
  if (int rc = device_info(&dev)) return rc;
  AttentionArgs a = {};
  a.c = c;
  a.q = query;
  a.q.max_q = std::min(query.max_q, query.n_rows);
  a.status = d_status;
  a.wait_ns = gather_wait_limit_ns();
  a.withhold = withhold_plans();
  // tokens that a list can name, in whole tiles
  const int64_t most = std::min<int64_t>(pages, c.table_cols) * c.page_tokens;
  a.score_cols = (int)((most + TILE - 1) / TILE * TILE);
  a.part = static_cast<float *>(d_scratch);
  a.columns = d_columns;
  a.pages = (int)pages;
  for (a.b0 = 0; a.b0 < c.batch; a.b0 += MAX_BATCH) {
    a.batch = std::min(c.batch - a.b0, MAX_BATCH);
    if (int rc = c.head_dim == 64 ? launch_types<64>(a, dev, s) : launch_types<128>(a, dev, s)) return rc;
  }
  return IBP_OK;
}

}  // namespace ibp
