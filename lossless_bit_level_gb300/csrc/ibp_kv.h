// Internal declarations of the 8-bit paged key/value cache (host side).
#pragma once

#include "ibp_internal.h"

namespace ibp {

constexpr int64_t KV_MAX_CAPACITY = int64_t(1) << 30;

int launch_kv_append(const ibp_kv_cache &c, const ibp_kv_rows &r, int32_t *d_new_lens,
                     int32_t *d_status, cudaStream_t s);
int launch_kv_read(const ibp_kv_cache &c, const int32_t *d_begin, int64_t n_out, void *k_out,
                   void *v_out, int dtype, int32_t *d_status, cudaStream_t s);
size_t kv_attention_scratch_bytes(const ibp_kv_cache &c, int64_t n_rows, int64_t max_q,
                                  int q_heads, bool with_weights);
int launch_kv_attention(const ibp_kv_cache &c, const ibp_kv_query &q, void *d_scratch,
                        int32_t *d_status, cudaStream_t s);
// Many query rows a sequence (ibp_kv_prefill.cu); no weights.
size_t kv_prefill_scratch_bytes(const ibp_kv_cache &c);
int launch_kv_prefill(const ibp_kv_cache &c, const ibp_kv_query &q, void *d_scratch,
                      int32_t *d_status, cudaStream_t s);
size_t kv_evict_scratch_bytes(const ibp_kv_cache &c, int64_t budget);
int launch_kv_evict(const ibp_kv_cache &c, const float *d_weights, int64_t weights_stride,
                    int64_t budget, int64_t recent, const ibp_kv_cache &dst, int32_t *d_new_lens,
                    float *d_new_weights, int64_t new_weights_stride, int32_t *d_kept,
                    void *d_scratch, int32_t *d_status, cudaStream_t s);

}  // namespace ibp
