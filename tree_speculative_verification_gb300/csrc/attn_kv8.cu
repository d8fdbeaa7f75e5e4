// attn_kv8.cu -- tree attention over the 8-bit KV cache.
//
// TreeAttention(u) = Attention(S_u) (SpecInfer, arXiv 2305.09781, Def. 4.1) with
// keys and values code * scale, and grouped query heads.
#include <math.h>

#include "kv8.cuh"

namespace ts {
namespace {

struct Attn8Args {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    const uint8_t *k8, *v8;
    const float *k_scale, *v_scale;
    const int32_t *prefix_len;
    ts_tree t;
    int Hq, H, G, rows;
    float scale_log2;
    PagedArgs pg;
    uint32_t *status;
};

constexpr int kWarps = 8;

// A warp per (node, query head): 32 keys at a time, lane j the score of key j,
// then the lanes share the value dims. Simple, and right for every size.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) k_attn_kv8_rows(Attn8Args a) {
    constexpr int DPL = D / 32;
    __shared__ float q_s[kWarps][D];
    const int b = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int n = a.t.n_nodes[b], P = a.prefix_len[b];
    const int r = blockIdx.x * kWarps + warp, i = r / a.G, hq = h * a.G + r % a.G;
    if (n <= 0 || i >= n) return;
    if (n > a.t.n_max || P < 0 || P > a.rows - n) {
        if (lane == 0 && h == 0 && r == 0) flag(a.status, TS_STATUS_INDEX);
        return;
    }
    const int v = a.t.perm[(size_t)b * a.t.n_max + i];
    if (v < 0 || v >= a.t.n_max) return;
    const size_t at = (((size_t)b * a.t.n_max + v) * a.Hq + hq) * D;
    for (int e = lane; e < D; e += 32) q_s[warp][e] = __bfloat162float(a.q[at + e]) * a.scale_log2;
    __syncwarp();
    float m = -INFINITY, l = 0.f, o[DPL] = {};
    const int L = P + n;
    for (int j0 = 0; j0 < L; j0 += 32) {
        const int j = j0 + lane;
        bool see = j < P;
        if (!see && j < L) see = j - P <= i && i < a.t.sub_end[(size_t)b * a.t.n_max + j - P];
        long long row = -1;
        if (j < L) row = cache_row(a.pg, b, h, a.H, a.rows, j);
        if (j < L && row < 0) flag(a.status, TS_STATUS_INDEX);
        float s = 0.f;
        if (row >= 0 && see) {
            const uint16_t *k = reinterpret_cast<const uint16_t *>(a.k8 + (size_t)row * D);
            for (int e = 0; e < D / 2; ++e) {
                const float2 f = fp8x2_to_float2(k[e]);
                s = fmaf(q_s[warp][2 * e], f.x, s);
                s = fmaf(q_s[warp][2 * e + 1], f.y, s);
            }
            s *= a.k_scale[row];
        }
        if (!see) s = -INFINITY;
        float mx = s;
        for (int o2 = 16; o2; o2 >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o2));
        const float mn = fmaxf(m, mx), alpha = mn > -INFINITY ? exp2f(m - mn) : 1.f;
        const float p = see ? exp2f(s - mn) : 0.f;
        m = mn;
        l = l * alpha + p;
        for (int e = 0; e < DPL; ++e) o[e] *= alpha;
        const float pv = see && row >= 0 ? p * a.v_scale[row] : 0.f;
        for (int k = 0; k < 32 && j0 + k < L; ++k) {
            const long long rk = __shfl_sync(~0u, row, k);
            const float pk = __shfl_sync(~0u, pv, k);
            const bool sk = __shfl_sync(~0u, (int)see, k);
            if (rk < 0 || !sk) continue;
            const uint8_t *vp = a.v8 + (size_t)rk * D + lane * DPL;
            for (int e = 0; e < DPL; e += 2) {
                const float2 f = fp8x2_to_float2(*reinterpret_cast<const uint16_t *>(vp + e));
                o[e] = fmaf(pk, f.x, o[e]);
                o[e + 1] = fmaf(pk, f.y, o[e + 1]);
            }
        }
    }
    for (int o2 = 16; o2; o2 >>= 1) l += __shfl_xor_sync(~0u, l, o2);
    for (int e = 0; e < DPL; ++e) a.out[at + lane * DPL + e] = __float2bfloat16(o[e] / l);
}

}  // namespace

size_t kv8_attention_ws_bytes(int, int, int, int, int, int) { return 256; }

cudaError_t launch_attn_kv8(void *out, const void *q, const ts_kv8 &kv, int Hq, const int32_t *prefix_len,
                            const ts_tree &t, float scale, void *, uint32_t *status, cudaStream_t s, const char **) {
    Attn8Args a = {(__nv_bfloat16 *)out, (const __nv_bfloat16 *)q, kv.k, kv.v, kv.k_scale, kv.v_scale, prefix_len, t,
                   Hq, kv.H, Hq / kv.H, kv8_rows(kv), scale * 1.4426950408889634f, kv8_pages(kv), status};
    const dim3 grid((t.n_max * a.G + kWarps - 1) / kWarps, kv.H, t.B), block(kWarps * 32);
    return kv.d == 128 ? launch(k_attn_kv8_rows<128>, grid, block, 0, s, a)
                       : launch(k_attn_kv8_rows<64>, grid, block, 0, s, a);
}

}  // namespace ts
