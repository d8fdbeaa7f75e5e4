// attn_decode.cu -- attention of one new token a request over its pages.
#include <cuda_bf16.h>
#include <math.h>

#include "decode.cuh"

namespace ts {
namespace {

constexpr int kDecodeWarps = 8;

// A CTA a (query head, request); each warp takes every kDecodeWarps-th key with
// a running maximum and sum of its own, joined at the end.
template <int D>
__global__ void __launch_bounds__(kDecodeWarps * 32)
k_attn_decode(__nv_bfloat16 *out, const __nv_bfloat16 *q, long long q_stride, const __nv_bfloat16 *kp,
              const __nv_bfloat16 *vp, const int32_t *bt, const int32_t *kv_len, int Hkv, int num_pages, int max_pages,
              float scale_log2, uint32_t *status) {
    constexpr int E = D / 32;
    __shared__ float m_s[kDecodeWarps], l_s[kDecodeWarps], o_s[kDecodeWarps][D];
    const int h = blockIdx.x, b = blockIdx.y, Hq = gridDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int n = kv_len[b];
    if (n < 0 || n > (long long)max_pages * TS_PAGE_KEYS) {
        if (threadIdx.x == 0) flag(status, TS_STATUS_INDEX);
        return;
    }
    float x[E], o[E] = {}, m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) x[e] = __bfloat162float(q[b * q_stride + (long long)h * D + lane * E + e]) * scale_log2;
    for (int j = warp; j < n; j += kDecodeWarps) {
        const int page = bt[(size_t)b * max_pages + j / TS_PAGE_KEYS];
        const bool ok = page >= 0 && page < num_pages;
        if (!ok && lane == 0) flag(status, TS_STATUS_INDEX);
        const size_t at = ok ? (((size_t)page * Hkv + h / (Hq / Hkv)) * TS_PAGE_KEYS + j % TS_PAGE_KEYS) * D + lane * E : 0;
        float s = 0.f;
        for (int e = 0; e < E; ++e) s += ok ? x[e] * __bfloat162float(kp[at + e]) : 0.f;
        for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(~0u, s, i);
        const float m1 = fmaxf(m, s), f = m == -INFINITY ? 1.f : exp2f(m - m1), p = s == -INFINITY ? 0.f : exp2f(s - m1);
        m = m1;
        l = l * f + p;
        for (int e = 0; e < E; ++e) o[e] = o[e] * f + (ok ? p * __bfloat162float(vp[at + e]) : 0.f);
    }
    if (lane == 0) m_s[warp] = m, l_s[warp] = l;
    for (int e = 0; e < E; ++e) o_s[warp][lane * E + e] = o[e];
    __syncthreads();
    if (threadIdx.x >= D) return;
    float top = -INFINITY, sum = 0.f, acc = 0.f;
    for (int w = 0; w < kDecodeWarps; ++w) top = fmaxf(top, m_s[w]);
    for (int w = 0; w < kDecodeWarps; ++w) {
        const float f = m_s[w] == -INFINITY ? 0.f : exp2f(m_s[w] - top);
        sum += l_s[w] * f;
        acc += o_s[w][threadIdx.x] * f;
    }
    out[((size_t)b * Hq + h) * D + threadIdx.x] = __float2bfloat16(n ? acc / sum : 0.f);
}

}  // namespace

size_t decode_ws_bytes(int B, int Hq, int Hkv, int d) { return 256; }

cudaError_t launch_attn_decode(void *out, const void *q, long long q_stride, const ts_paged_kv &kv,
                               const int32_t *kv_len, int B, int Hq, int Hkv, int d, float scale, void *ws,
                               uint32_t *status, cudaStream_t s) {
    auto go = [&](auto kern) {
        return launch(kern, dim3(Hq, B), dim3(kDecodeWarps * 32), 0, s, (__nv_bfloat16 *)out, (const __nv_bfloat16 *)q,
                      q_stride, (const __nv_bfloat16 *)kv.k_pages, (const __nv_bfloat16 *)kv.v_pages, kv.block_table,
                      kv_len, Hkv, (int)kv.num_pages, (int)kv.max_pages, scale * 1.4426950408889634f, status);
    };
    return d == 128 ? go(k_attn_decode<128>) : go(k_attn_decode<64>);
}

}  // namespace ts
