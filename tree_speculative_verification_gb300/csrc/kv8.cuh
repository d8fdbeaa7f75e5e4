// kv8.cuh -- internals of the 8-bit KV cache (e4m3 codes, one fp32 scale per
// row and head) and of the head norms with rotation.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ts_internal.cuh"

namespace ts {

constexpr float kFp8Max = 448.f;                       // largest e4m3 value
constexpr float kScaleMin = 7.888609052210118e-31f;    // 2^-100: scales stay normal, 1 / scale finite
constexpr float kLog2e = 1.4426950408889634f;

inline PagedArgs kv8_pages(const ts_kv8 &kv) {
    PagedArgs pg;
    pg.bt = kv.block_table;
    pg.max_pages = kv.max_pages;
    pg.num_pages = kv.num_pages;
    return pg;
}
inline int kv8_rows(const ts_kv8 &kv) { return kv.block_table ? kv.max_pages * TS_PAGE_KEYS : kv.L_max; }

// Two e4m3 codes as fp32 (exact).
__device__ __forceinline__ float2 fp8x2_to_float2(uint16_t c) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3);
    return __half22float2(__half2(h));
}

cudaError_t launch_qk_norm_rope(void *q_out, void *k_out, const void *q, const void *k, int Hq, int Hk, int d,
                                long long q_stride, long long k_stride, const ts_qk_rope &rope, const ts_tree &t,
                                ts_dtype dt, cudaStream_t s);
cudaError_t launch_kv8_append(const ts_kv8 &kv, const void *k_new, const void *v_new, long long k_stride,
                              long long v_stride, const ts_qk_rope *rope, void *q_out, const void *q, int Hq,
                              long long q_stride, const int32_t *prefix_len, const ts_tree &t, ts_dtype dt,
                              uint32_t *status, cudaStream_t s);
cudaError_t launch_kv8_read(void *k_out, void *v_out, const ts_kv8 &kv, const int32_t *row_begin,
                            const int32_t *row_end, int L_out, ts_dtype dt, uint32_t *status, cudaStream_t s);
cudaError_t launch_kv8_commit(const ts_kv8 &kv, const int32_t *prefix_len, int32_t *new_prefix_len,
                              const int32_t *out_path, const int32_t *out_count, const ts_tree &t, uint32_t *status,
                              cudaStream_t s);

size_t kv8_attention_ws_bytes(int B, int Hq, int Hkv, int n_max, int d, int L_max);
cudaError_t launch_attn_kv8(void *out, const void *q, const ts_kv8 &kv, int Hq, const int32_t *prefix_len,
                            const ts_tree &t, float scale, void *ws, uint32_t *status, cudaStream_t s,
                            const char **why);

}  // namespace ts
