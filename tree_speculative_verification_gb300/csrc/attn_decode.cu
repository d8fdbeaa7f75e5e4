// attn_decode.cu -- attention of one new token a request over its pages.
//
// A step over 16 keys is two small products on the tensor cores with the keys
// (then the head's dims) as the 16 rows and up to 8 query heads of one
// key/value head as the columns: S^T = K Q^T, O^T += V^T P^T (mma.sync
// m16n8k16). Bound by the cache's bytes: 1 to 16 flops a byte, where tcgen05,
// whose tiles have 128 rows at least and come from shared memory, would add a
// trip through it and nothing else. So K and V go from global memory into the
// registers that the products read them from, with no stop on the way: which 16
// keys are a step's rows, and which dims a product's k index means, is free, and
// is chosen so that each lane's part of a step is whole 16-byte pieces.
//
// The work is cut evenly: the tiles (64 keys, a page) of all (request, key/value
// head, block of query heads) items stand in one line, and every CTA takes an
// equal stretch of it, found from the lengths on the GPU. An item that lies in
// several CTAs' stretches leaves a part (O, maximum, sum) of each in the
// workspace, and the CTA that finds by a counter that it is the item's last one
// joins them, in their order, so that results do not depend on which that is.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "attn_common.cuh"
#include "decode.cuh"

namespace ts {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kRoom = 8.f;   // how far (in powers of 2) a score may pass the running maximum before that is raised

struct DecodeArgs {
    __nv_bfloat16 *out;
    const uint4 *q, *k, *v;
    long long q_stride;   // in 16-byte pieces
    const int32_t *bt, *kv_len;
    int B, Hq, Hkv, G, blocks;   // query heads a key/value head; blocks of them
    int num_pages, max_pages;
    float scale_log2;
    unsigned *counters;   // [grid]: parts of the item that starts in a CTA's stretch and ends in a later one's
    float *parts;         // [grid][2][heads][D + 2]
    uint32_t *status;
};

__device__ __forceinline__ uint4 ld_stream(const uint4 *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 block of 16-bit numbers transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t part_of(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ float guarded(float m) { return m == -INFINITY ? 0.f : m; }

// CTAs an SM, as the registers allow.
template <int D, int NT>
constexpr int kPerSm = D == 64 ? (NT == 1 ? 4 : 3) : (NT == 1 ? 3 : 2);

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, kPerSm<D, NT>) k_attn_decode(DecodeArgs a) {
    constexpr int HB = 8 * NT;           // query heads of a block
    constexpr int VEC = D / 8;           // 16-byte pieces of a row
    constexpr int KC = D / 32, VC = D / 64;
    constexpr int ROW = D + 4;           // floats between heads in shared memory
    __shared__ float o_s[kWarps][HB][ROW];
    __shared__ float m_s[kWarps][HB], l_s[kWarps][HB];
    __shared__ long long sum_s[kWarps], first_s;
    __shared__ int len_s[kThreads], req_s, last_s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    pdl_wait();
    pdl_trigger();

    // ---- the plan: which stretch of the line of tiles is this CTA's
    auto pages_of = [&](int b, int n) {
        if (n < 0 || n > (long long)a.max_pages * TS_PAGE_KEYS) {
            if (blockIdx.x == 0) flag(a.status, TS_STATUS_INDEX);
            return 0;
        }
        return (n + TS_PAGE_KEYS - 1) / TS_PAGE_KEYS;
    };
    auto block_sum = [&](long long v, long long &before) {   // before: of the threads before this one
        long long run = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += y;
        }
        __syncthreads();
        if (lane == 31) sum_s[warp] = run;
        __syncthreads();
        long long all = 0;
        before = run - v;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sum_s[w];
            all += sum_s[w];
        }
        return all;
    };
    const int items = a.Hkv * a.blocks;   // of a request
    long long mine = 0, before = 0;
    for (int b = tid; b < a.B; b += kThreads) {
        const int n = a.kv_len[b];
        if (b < kThreads) len_s[b] = n;
        mine += pages_of(b, n);
    }
    for (int b = blockIdx.x; b < a.B; b += gridDim.x)   // no key: zeros
        if (a.kv_len[b] == 0)
            for (int i = tid; i < a.Hq * VEC; i += kThreads)
                ((uint4 *)a.out)[(size_t)b * a.Hq * VEC + i] = make_uint4(0, 0, 0, 0);
    const long long T = block_sum(mine, before) * items;
    const long long ctas = min((long long)gridDim.x, T), c = blockIdx.x;
    if (c >= ctas) return;
    long long x = T * c / ctas;
    const long long x_end = T * (c + 1) / ctas;
    for (long long base = 0, done = 0; base < a.B; base += kThreads) {
        const int b = (int)base + tid, p = b < a.B ? pages_of(b, a.kv_len[b]) : 0;
        const long long all = block_sum(p, before);
        if ((done + before) * items <= x && x < (done + before + p) * items) req_s = b, first_s = (done + before) * items;
        done += all;
        if (x < done * items) break;
    }
    __syncthreads();
    int b = req_s;
    long long first = first_s;             // the line's tile at which request b starts

    while (x < x_end) {
        const int n = b < kThreads ? len_s[b] : a.kv_len[b], pages = pages_of(b, n);
        if (pages == 0 || x >= first + (long long)pages * items) {
            first += (long long)pages * items;
            ++b;
            continue;
        }
        const int item = (int)((x - first) / pages), kvh = item / a.blocks, h0 = (item - kvh * a.blocks) * HB;
        const long long i0 = first + (long long)item * pages, i1 = i0 + pages, x1 = min(i1, x_end);
        const int step0 = (int)(x - i0) * (TS_PAGE_KEYS / 16),
                  step1 = min((int)(x1 - i0) * (TS_PAGE_KEYS / 16), (n + 15) / 16);
        const int32_t *bt = a.bt + (size_t)b * a.max_pages;

        // ---- a step's loads. Lane (g, t) takes of K rows g and g + 8, pieces t, t + 4, ..; of V rows 2t, 2t + 1, 2t + 8,
        // 2t + 9, pieces g, g + 8
        uint4 kr[2][KC], vr[4][VC], qr[NT][KC];
        const uint4 zero = make_uint4(0, 0, 0, 0);
        auto page_of = [&](int s) { return s < step1 ? __ldg(bt + (s >> 2)) : 0; };
        auto rows_at = [&](int page, int s) { return ((size_t)page * a.Hkv + kvh) * TS_PAGE_KEYS + (s & 3) * 16; };
        auto is_page = [&](int page) {
            const bool ok = page >= 0 && page < a.num_pages;
            if (!ok) flag(a.status, TS_STATUS_INDEX);
            return ok;
        };
        auto load_k = [&](int s, int page, bool ok) {
            const uint4 *p = a.k + rows_at(page, s) * VEC + t;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int i = 0; i < KC; ++i)
                    kr[r][i] = ok && s * 16 + g + 8 * r < n ? ld_stream(p + (g + 8 * r) * VEC + 4 * i) : zero;
        };
        auto load_v = [&](int s, int page, bool ok) {
            const uint4 *p = a.v + rows_at(page, s) * VEC + g;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 2 * t + (r & 1) + 8 * (r >> 1);
#pragma unroll
                for (int i = 0; i < VC; ++i) vr[r][i] = ok && s * 16 + row < n ? ld_stream(p + row * VEC + 8 * i) : zero;
            }
        };
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int h = h0 + 8 * j + g;
            const uint4 *p = a.q + b * a.q_stride + (size_t)(kvh * a.G + h) * VEC + t;
#pragma unroll
            for (int i = 0; i < KC; ++i) qr[j][i] = h < a.G ? __ldg(p + 4 * i) : zero;
        }
        float o[NT][VEC / 2][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            m[j][0] = m[j][1] = -INFINITY;
            l[j][0] = l[j][1] = 0.f;
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
        }
        int s = step0 + warp;
        int page_v = page_of(s), page = page_of(s + kWarps);   // of the step whose V is loaded next; of the one after it
        bool ok_v = s < step1 && is_page(page_v), ok;
        if (s < step1) {
            load_k(s, page_v, ok_v);
            load_v(s, page_v, ok_v);
        }
        for (; s < step1; s += kWarps) {
            float p[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                p[j][0] = p[j][1] = p[j][2] = p[j][3] = 0.f;
#pragma unroll
                for (int i = 0; i < KC; ++i) {
                    mma(p[j], kr[0][i].x, kr[1][i].x, kr[0][i].y, kr[1][i].y, qr[j][i].x, qr[j][i].y);
                    mma(p[j], kr[0][i].z, kr[1][i].z, kr[0][i].w, kr[1][i].w, qr[j][i].z, qr[j][i].w);
                }
            }
            const int next = s + kWarps;
            page_v = page;
            ok = next < step1 && is_page(page);
            if (next < step1) load_k(next, page, ok);
            page = page_of(next + kWarps);
            // scores as exponents of 2; keys behind the last one have none
            bool raise = false;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[j][e] = s * 16 + g + 8 * (e >> 1) < n ? p[j][e] * a.scale_log2 : -INFINITY;
                    raise |= p[j][e] > m[j][e & 1] + kRoom;
                }
            if (__any_sync(~0u, raise)) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(p[j][e], p[j][e + 2]);
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, 8));
                        top = fmaxf(m[j][e], fmaxf(top, __shfl_xor_sync(~0u, top, 16)));
                        const float f = ex2(m[j][e] - guarded(top));
                        m[j][e] = top;
                        l[j][e] *= f;
#pragma unroll
                        for (int i = 0; i < VEC / 2; ++i) o[j][i][e] *= f, o[j][i][e + 2] *= f;
                    }
            }
            // P^T as the second factor, in two bf16 numbers: the upper half of the fp32 number, and what is left, rounded
            // (in all 16 bits of each weight). What is left counts as 2^-126 at least, so that an infinite value comes
            // through as one
            uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[j][e] = ex2(p[j][e] - guarded(m[j][e & 1]));
                    l[j][e & 1] += p[j][e];
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float p0 = p[j][2 * r], p1 = p[j][2 * r + 1];
                    const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
                    hi[j][r] = transposed(__byte_perm(u0, u1, 0x7632));
                    const __nv_bfloat162 rest =
                        __floats2bfloat162_rn(fmaxf(p0 - __uint_as_float(u0 & 0xffff0000u), 1.17549435e-38f),
                                              fmaxf(p1 - __uint_as_float(u1 & 0xffff0000u), 1.17549435e-38f));
                    lo[j][r] = transposed(*reinterpret_cast<const uint32_t *>(&rest));
                }
            }
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {   // dims 8 g + 2 (i % 4) and the next one, of piece g + 8 (i / 4)
                const uint32_t w0 = part_of(vr[0][i / 4], i % 4), w1 = part_of(vr[1][i / 4], i % 4),
                               w2 = part_of(vr[2][i / 4], i % 4), w3 = part_of(vr[3][i / 4], i % 4);
                const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632),
                               a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    mma(o[j][i], a0, a1, a2, a3, hi[j][0], hi[j][1]);
                    mma(o[j][i], a0, a1, a2, a3, lo[j][0], lo[j][1]);
                }
            }
            if (next < step1) load_v(next, page_v, ok);
        }

        // ---- the CTA's warps joined
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = 8 * j + 2 * t + e;
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) l[j][e] += __shfl_xor_sync(~0u, l[j][e], k);
                if (g == 0) m_s[warp][h] = m[j][e], l_s[warp][h] = l[j][e];
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i)
                    *reinterpret_cast<float2 *>(&o_s[warp][h][64 * (i / 4) + 8 * g + 2 * (i % 4)]) =
                        make_float2(o[j][i][e], o[j][i][e + 2]);
            }
        __syncthreads();
        const bool whole = x == i0 && x1 == i1;
        float *part = a.parts + (size_t)(2 * c + (x == i0)) * HB * (D + 2);
        for (int q = tid; q < HB * D / 4; q += kThreads) {
            const int h = q / (D / 4), dd = q % (D / 4) * 4;
            if (h0 + h >= a.G) break;
            float top = -INFINITY, sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w][h]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(m_s[w][h] - guarded(top));
                const float4 y = *reinterpret_cast<const float4 *>(&o_s[w][h][dd]);
                sum = fmaf(l_s[w][h], f, sum);
                acc.x = fmaf(y.x, f, acc.x), acc.y = fmaf(y.y, f, acc.y), acc.z = fmaf(y.z, f, acc.z), acc.w = fmaf(y.w, f, acc.w);
            }
            if (whole) {
                const float f = 1.f / sum;
                __nv_bfloat162 r0 = __floats2bfloat162_rn(acc.x * f, acc.y * f), r1 = __floats2bfloat162_rn(acc.z * f, acc.w * f);
                *reinterpret_cast<uint2 *>(a.out + ((size_t)b * a.Hq + kvh * a.G + h0 + h) * D + dd) =
                    make_uint2(*reinterpret_cast<uint32_t *>(&r0), *reinterpret_cast<uint32_t *>(&r1));
            } else {
                *reinterpret_cast<float4 *>(part + h * D + dd) = acc;
                if (dd == 0) part[HB * D + h] = top, part[HB * (D + 1) + h] = sum;
            }
        }
        if (!whole) {
            // ---- the item's CTAs c0 .. c1 joined by the one that comes here last
            const long long c0 = ((i0 + 1) * ctas - 1) / T, c1 = (i1 * ctas - 1) / T;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                last_s = atomicAdd(a.counters + c0, 1u) == c1 - c0;
                if (last_s) a.counters[c0] = 0;
                __threadfence();
            }
            __syncthreads();
            if (last_s) {
                for (int q = tid; q < HB * D / 4; q += kThreads) {
                    const int h = q / (D / 4), dd = q % (D / 4) * 4;
                    if (h0 + h >= a.G) break;
                    float top = -INFINITY, sum = 0.f;
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    auto part_at = [&](long long k) { return a.parts + (size_t)(2 * k + (k == c0)) * HB * (D + 2); };
#pragma unroll 8
                    for (long long k = c0; k <= c1; ++k) top = fmaxf(top, __ldcg(part_at(k) + HB * D + h));
#pragma unroll 8
                    for (long long k = c0; k <= c1; ++k) {
                        const float *y = part_at(k);
                        const float f = ex2(__ldcg(y + HB * D + h) - guarded(top));
                        const float4 v = __ldcg(reinterpret_cast<const float4 *>(y + h * D + dd));
                        sum = fmaf(__ldcg(y + HB * (D + 1) + h), f, sum);
                        acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y), acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
                    }
                    const float f = 1.f / sum;
                    __nv_bfloat162 r0 = __floats2bfloat162_rn(acc.x * f, acc.y * f), r1 = __floats2bfloat162_rn(acc.z * f, acc.w * f);
                    *reinterpret_cast<uint2 *>(a.out + ((size_t)b * a.Hq + kvh * a.G + h0 + h) * D + dd) =
                        make_uint2(*reinterpret_cast<uint32_t *>(&r0), *reinterpret_cast<uint32_t *>(&r1));
                }
            }
        }
        __syncthreads();   // shared memory is the next item's
        x = x1;
    }
}

int grid_of(int d, int HB) {
    return num_sms() * (d == 64 ? (HB == 8 ? kPerSm<64, 1> : kPerSm<64, 2>) : (HB == 8 ? kPerSm<128, 1> : kPerSm<128, 2>));
}
int heads_of(int G) { return G > 8 ? 16 : 8; }
size_t counter_bytes() { return ((size_t)num_sms() * kPerSm<64, 1> * 4 + 255) / 256 * 256; }   // the largest grid's

}  // namespace

// Counters first: one workspace serves calls of several sizes.
size_t decode_ws_bytes(int B, int Hq, int Hkv, int d) {
    const int HB = heads_of(Hq / Hkv);
    return counter_bytes() + (size_t)grid_of(d, HB) * 2 * HB * (d + 2) * 4;
}

cudaError_t launch_attn_decode(void *out, const void *q, long long q_stride, const ts_paged_kv &kv,
                               const int32_t *kv_len, int B, int Hq, int Hkv, int d, float scale, void *ws,
                               uint32_t *status, cudaStream_t s) {
    const int G = Hq / Hkv, HB = heads_of(G);
    const DecodeArgs a{(__nv_bfloat16 *)out,
                       (const uint4 *)q,
                       (const uint4 *)kv.k_pages,
                       (const uint4 *)kv.v_pages,
                       q_stride / 8,
                       kv.block_table,
                       kv_len,
                       B,
                       Hq,
                       Hkv,
                       G,
                       (G + HB - 1) / HB,
                       kv.num_pages,
                       kv.max_pages,
                       scale * 1.4426950408889634f,
                       (unsigned *)ws,
                       (float *)((char *)ws + counter_bytes()),
                       status};
    auto go = [&](auto kern) { return launch(kern, dim3(grid_of(d, HB)), dim3(kThreads), 0, s, a); };
    if (d == 128) return HB == 8 ? go(k_attn_decode<128, 1>) : go(k_attn_decode<128, 2>);
    return HB == 8 ? go(k_attn_decode<64, 1>) : go(k_attn_decode<64, 2>);
}

}  // namespace ts
