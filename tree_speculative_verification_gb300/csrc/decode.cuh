// decode.cuh -- internals of a decode step on the paged cache: pages and slots,
// rows by slot, attention of one new token a request, and token sampling.
#pragma once
#include "ts_internal.cuh"

namespace ts {

cudaError_t launch_pages_build(const ts_page_pool &pool, int32_t *new_held, int32_t *new_state, int32_t *slot,
                               int max_slots, int32_t *slot_offset, const int32_t *row_begin, const int32_t *row_end,
                               uint32_t *status, cudaStream_t s);
cudaError_t launch_append_slots(const ts_paged_kv &kv, const void *k_new, const void *v_new, long long k_stride,
                                long long v_stride, const int32_t *slot, int T, int H, int d, uint32_t *status,
                                cudaStream_t s);

size_t decode_ws_bytes(int B, int Hq, int Hkv, int d);
cudaError_t launch_attn_decode(void *out, const void *q, long long q_stride, const ts_paged_kv &kv,
                               const int32_t *kv_len, int B, int Hq, int Hkv, int d, float scale, void *ws,
                               uint32_t *status, cudaStream_t s);

// One row's settings are looked up in the arrays that are not null.
struct SampleArgs {
    int32_t *token;
    float *probs, *kept;
    const void *logits;
    long long stride;
    const float *u, *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p;
    int R, V;
    uint32_t *status;
};
cudaError_t launch_sample(const SampleArgs &a, ts_dtype dt, cudaStream_t s);

}  // namespace ts
