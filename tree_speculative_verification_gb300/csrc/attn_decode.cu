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
// equal stretch of it, found from the lengths on the GPU (or, where there are more
// CTAs than items, one part of one item). An item that lies in
// several CTAs' stretches leaves a part (O, maximum, sum) of each in the
// workspace, and the CTA that finds by a counter that it is the item's last one
// joins them, in their order, so that results do not depend on which that is.
//
// 64 requests of 1024 keys, 56 heads: 277 us, the copy rate; 4 of 16384 keys,
// 64 heads over 8: 46 us, of which the stream takes 38 (the copy rate again), launch
// and plan 4, the join 4; 8 of 2048 keys, 32 over 8: 17 us, of which the stream
// takes 9.5. One request's start is plan, loads, sums: 4.4 us.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>

#include "attn_common.cuh"
#include "decode.cuh"

namespace ts {
namespace {

constexpr float kRoom = 8.f;   // how far (in powers of 2) a score may pass the running maximum before that is raised

struct DecodeArgs {
    __nv_bfloat16 *out;
    const uint4 *q, *k, *v;
    long long q_stride;   // in 16-byte pieces
    const int32_t *bt, *kv_len;
    int B, Hq, Hkv, G, blocks;   // query heads a key/value head; blocks of them
    int num_pages, max_pages;
    float scale_log2;
    unsigned *counters;   // [2][grid]: parts there are of the item (the group of parts) that starts in a CTA's stretch
    float *parts;         // [grid][2][heads][D + 2]
    uint32_t *status;
};

// 16 bytes that are read once, or zeros where yes is false (no branch: the loads of a step are one run of instructions).
__device__ __forceinline__ uint4 ld_stream(const uint4 *p, bool yes) {
    uint4 v;
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %5, 0;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n mov.u32 %3, 0;\n"
        " @p ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n}\n"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(p), "r"((uint32_t)yes));
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

// As many warps an SM as the registers allow, in CTAs of four, or all in one CTA where there are few items: the more warps
// share an item, the fewer parts of it are joined through the workspace, but the more of them wait for one another at its
// end. In fours and in one: one request of 16384 keys, 8 heads 21.4 and 17.6 us; 8 requests of 2048 keys, 8 heads 16.8 and
// 19.0; 64 requests of 1024 keys, 56 heads 276 and 296.
template <int D, int NT>
constexpr int kFours = D == 64 ? (NT == 1 ? 4 : 3) : (NT == 1 ? 3 : 2);
template <int D, int NT, bool ONE>
constexpr int kWarps = ONE ? 4 * kFours<D, NT> : 4;
template <int D, int NT, bool ONE>
constexpr int kPerSm = ONE ? 1 : kFours<D, NT>;
template <int D, int NT, bool ONE>
constexpr int kSmem = kWarps<D, NT, ONE> * 8 * NT * (D + 4) * 4;
constexpr int kFewItems = 48;

// A stretch of one item's keys: steps [step0, step1) of 16 keys.
struct Segment {
    int b, n, kvh, h0;   // request, its keys, key/value head, first query head of the block
    int step0, step1;
    int i0, i1, x1;      // the item's tiles in the line, and where the segment ends
    const int32_t *bt;
};
// An item in several CTAs' stretches, from c0 on: whose rows it is, and what its parts are counted by.
struct Shared {
    int b, kvh, h0;
    int c0, k0;          // the item's first CTA, the group's
    int n, groups;       // parts to be counted at k0, groups (0: one level)
};

constexpr int kGroup = 16, kGroupFrom = 33;   // parts are joined in two levels, kGroup at a time, from kGroupFrom on
constexpr int kFewParts = 8;
constexpr int kMostParts = 64, kMostCtas = kMostParts * kGroup - 1;   // parts, or groups, in one join; CTAs that allows

// Adds one to a counter: what the CTA has written before (behind a barrier) is seen by whoever finds it counted and
// then sees_counted(). The count is only waited for where it is used.
__device__ __forceinline__ unsigned count_up(unsigned *p) {
    unsigned old;
    asm volatile("atom.add.release.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
    return old;
}
__device__ __forceinline__ void sees_counted() { asm volatile("fence.acq_rel.gpu;" ::: "memory"); }

template <int D, int NT, bool ONE>
__global__ void __launch_bounds__(32 * kWarps<D, NT, ONE>, kPerSm<D, NT, ONE>) k_attn_decode(DecodeArgs a) {
    constexpr int W = kWarps<D, NT, ONE>, kThreads = 32 * W;
    constexpr int HB = 8 * NT;           // query heads of a block
    constexpr int VEC = D / 8;           // 16-byte pieces of a row
    constexpr int KC = D / 32, VC = D / 64;
    constexpr int ROW = D + 4;           // floats between heads in shared memory
    constexpr int PART = HB * (D + 2);   // floats of a part: O, maxima, sums
    extern __shared__ float smem[];
    float(*o_s)[HB][ROW] = reinterpret_cast<float(*)[HB][ROW]>(smem);   // [W]
    __shared__ float m_s[W][HB], l_s[W][HB], f_s[kMostParts][HB];
    __shared__ long long sum_s[W];
    __shared__ int len_s[kThreads], req_s, first_s, items_s[W], most_s[W], last_s, part_s[2];
    __shared__ Shared shared_s[2];   // of the CTA's first segment, of its last
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    pdl_wait();
    pdl_trigger();

    // ---- the plan: which stretch of the line of tiles is this CTA's
    auto pages_of = [&](int n) {
        if (n < 0 || n > (long long)a.max_pages * TS_PAGE_KEYS) return 0;
        return (n + TS_PAGE_KEYS - 1) / TS_PAGE_KEYS;
    };
    // sum over the CTA; before: over the threads before this one
    auto block_sum = [&](long long v, long long &before) {
        long long run = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, run, o);
            if (lane >= o) run += y;
        }
        if (lane == 31) sum_s[warp] = run;
        __syncthreads();
        long long all = 0;
        before = run - v;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < warp) before += sum_s[w];
            all += sum_s[w];
        }
        return all;
    };
    const int items = a.Hkv * a.blocks;   // of a request
    auto no_keys = [&](int b) {           // zeros
        for (int i = tid; i < a.Hq * VEC; i += kThreads)
            ((uint4 *)a.out)[(size_t)b * a.Hq * VEC + i] = make_uint4(0, 0, 0, 0);
    };
    // Up to 32 requests every warp plans for itself, a lane a request, without a barrier (one request of 100 keys 4.2 us, and 4.6
    // by all warps together).
    const bool few = a.B <= 32;
    int lane_n = 0, lane_p = 0, lane_to = 0;   // keys, pages, and pages up to and with this request
    long long mine = 0, before = 0, all_tiles;
    int live = 0, live_items = 0, mine_first = 0;
    int most_p = 0;
    bool alike = false;                        // all requests with keys have as many pages (more than 32 of them)
    if (few) {
        if (lane < a.B) lane_n = a.kv_len[lane];
        lane_p = lane_to = pages_of(lane_n);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(~0u, lane_to, o);
            if (lane >= o) lane_to += y;
        }
        live_items = __popc(__ballot_sync(~0u, lane_p > 0));
        most_p = __reduce_max_sync(~0u, lane_p);
        all_tiles = (long long)__shfl_sync(~0u, lane_to, 31) * items;
        if (blockIdx.x == 0 && warp == 0 && lane_p == 0 && lane_n != 0) flag(a.status, TS_STATUS_INDEX);
        for (int b = blockIdx.x; b < a.B; b += gridDim.x)
            if (__shfl_sync(~0u, lane_n, b) == 0) no_keys(b);
    } else {
        for (int b = tid; b < a.B; b += kThreads) {
            const int n = a.kv_len[b], p = pages_of(n);
            if (b < kThreads) len_s[b] = n, mine_first = p;
            mine += p;
            live += p > 0;
            most_p = max(most_p, p);
            if (p == 0 && n != 0 && blockIdx.x == 0) flag(a.status, TS_STATUS_INDEX);
        }
        for (int b = blockIdx.x; b < a.B; b += gridDim.x)
            if (a.kv_len[b] == 0) no_keys(b);
        live = __reduce_add_sync(~0u, live);
        most_p = __reduce_max_sync(~0u, most_p);
        if (lane == 0) items_s[warp] = live, most_s[warp] = most_p;
        all_tiles = block_sum(mine, before);
#pragma unroll
        for (int w = 0; w < W; ++w) live_items += items_s[w], most_p = max(most_p, most_s[w]);
        alike = all_tiles == (long long)live_items * most_p;
        all_tiles *= items;
    }
    if (all_tiles == 0 || all_tiles > INT32_MAX) {
        if (all_tiles && blockIdx.x == 0 && tid == 0) flag(a.status, TS_STATUS_INDEX);
        return;
    }
    const int T = (int)all_tiles, c = blockIdx.x;
    live_items *= items;
    // As many CTAs as the GPU holds. A part that has to be joined costs 2 to 3 us, a step of every warp 0.8 us: items of up to
    // kWhole tiles are not cut, and none into parts of less than a step of every warp. (Whole up to 3 steps of all twelve warps
    // or 4: one request of 768 keys, 8 heads 8.1 and 9.6 us; up to 2: of 512 keys 8.7 and 8.0. Up to 4 of four or 5: 8 requests
    // of 300 keys, 8 heads 9.1 and 10.8.)
    // Where there are enough CTAs each gets one part of one item, of at most so many tiles that the parts are no more than the
    // CTAs, unless that is kJoin, or a tenth, above an equal stretch of the line: no CTA then has parts of two items to leave.
    // (Such parts and equal stretches: 16 requests, 8 heads, of 300 keys 10.9 and 13.9 us, of 1500 21.6 and 23.4; 4 requests of
    // 16384 keys, 8 heads 46 and 48; 8 of 100 to 600 keys, 8 heads 9.5 and 14.0, 16 of 300 to 3000 25.2 and 26.1. By 20 steps of
    // every warp above it is too much: 29 requests of 2500 keys 60 and 51.) That is found by a lane a request; more requests
    // than a warp has lanes are cut into parts where they are all alike, or where that leaves out a tenth of the CTAs at most.
    constexpr int kWhole = (ONE ? 3 : 4) * W / 4, kLeast = W / 4, kJoin = 8 * W / 4;
    const int grid = gridDim.x;
    int ctas = grid, x = 0, x_end = 0, req = 0, first = 0;   // a request, and the line's tile at which it starts
    int parts = 0;                                           // of the CTA's one item (0: a stretch of the line)
    if (few && live_items <= grid) {
        auto parts_of = [&](int s) { return lane_p <= kWhole ? (lane_p > 0) : (int)((unsigned)(lane_p + s - 1) / (unsigned)s); };
        auto number = [&](int s) { return items * (int)__reduce_add_sync(~0u, parts_of(s)); };
        const bool same = __all_sync(~0u, lane_p == 0 || lane_p == most_p);
        const int share = T / grid;
        int s = share + max(kJoin, share / 10);
        bool fits = most_p <= kWhole;
        if (!fits && same) {
            const int fit = grid / live_items, need = max(kLeast, (most_p + fit - 1) / fit);
            fits = need <= s, s = need;
        } else if (!fits) {
            int lo = max(kLeast, share + (share * grid < T));
            // (a part more an item than its share of the line are CTAs enough)
            const int enough = grid > live_items ? (int)((unsigned)T / (unsigned)(grid - live_items)) + 1 : most_p;
            fits = enough <= s || number(s) <= grid;
            s = max(lo, min(s, enough));
#pragma unroll 1
            for (int i = 0; i < 3 && fits && lo < s; ++i) {
                const int m = (lo + s) / 2;
                if (number(m) <= grid) s = m;
                else lo = m + 1;
            }
        }
        if (fits) {
            const int own = parts_of(s);
            int to = own * items;                            // CTAs up to and with this request's
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(~0u, to, o);
                if (lane >= o) to += y;
            }
            if (c >= __shfl_sync(~0u, to, 31)) return;
            req = __ffs(__ballot_sync(~0u, to - own * items <= c && c < to)) - 1;
            const int at = c - __shfl_sync(~0u, to - own * items, req), pages = __shfl_sync(~0u, lane_p, req);
            parts = __shfl_sync(~0u, own, req), first = __shfl_sync(~0u, (lane_to - lane_p) * items, req);
            const int item = (unsigned)at / (unsigned)parts, k = at - item * parts, each = pages / parts, over = pages - each * parts;
            if (tid == 0) part_s[0] = c - k;                 // the first one's CTA
            x = first + item * pages + each * k + over * k / parts;
            x_end = first + item * pages + each * (k + 1) + over * (k + 1) / parts;
        }
    }
    if (!parts) {
        if (!few && live_items <= grid) {
            const int pages = T / live_items, most = pages <= kWhole ? 1 : pages / kLeast, fit = grid / live_items;
            if (most <= fit || grid % live_items <= grid / 10 || (alike && (pages + fit - 1) / fit <= T / grid + kJoin))
                ctas = min(most, fit) * live_items;
        }
        if (c >= ctas) return;
        const int q0 = T / ctas, r0 = T - q0 * ctas;
        auto stretch = [&](int c) { return q0 * c + (unsigned)(r0 * c) / (unsigned)ctas; };   // floor(T c / ctas)
        x = stretch(c), x_end = stretch(c + 1);
        if (few) {
            const int lo = (lane_to - lane_p) * items;
            req = __ffs(__ballot_sync(~0u, lo <= x && x < lo + lane_p * items)) - 1;
            first = __shfl_sync(~0u, lo, req);
        } else if (a.B <= kThreads) {
            const int lo = (int)before * items;
            if (lo <= x && x < lo + mine_first * items) req_s = tid, first_s = lo;
            __syncthreads();
        } else {
            int done = 0;
            for (int base = 0; base < a.B; base += kThreads) {
                const int b = base + tid, p = b < a.B ? pages_of(a.kv_len[b]) : 0;
                __syncthreads();
                const int all = (int)block_sum(p, before), lo = (done + (int)before) * items;
                if (lo <= x && x < lo + p * items) req_s = b, first_s = lo;
                done += all;
                if (x < done * items) break;
            }
            __syncthreads();
        }
        if (!few) req = req_s, first = first_s;
    }
    if (tid == 0) part_s[1] = parts;
    auto segment = [&](int x) {            // the one that starts at tile x, below x_end
        Segment z;
        int n, pages;
        while (true) {
            n = few ? __shfl_sync(~0u, lane_n, req) : req < kThreads ? len_s[req] : a.kv_len[req], pages = pages_of(n);
            if (x < first + pages * items) break;
            first += pages * items;
            ++req;
        }
        const int item = (unsigned)(x - first) / (unsigned)pages;
        z.b = req, z.n = n, z.kvh = a.blocks == 1 ? item : item / a.blocks, z.h0 = (item - z.kvh * a.blocks) * HB;
        z.i0 = first + item * pages, z.i1 = z.i0 + pages, z.x1 = min(z.i1, x_end);
        z.step0 = (x - z.i0) * (TS_PAGE_KEYS / 16);
        z.step1 = min((z.x1 - z.i0) * (TS_PAGE_KEYS / 16), (n + 15) / 16);
        z.bt = a.bt + (size_t)req * a.max_pages;
        return z;
    };

    // ---- a step's loads. Lane (g, t) takes of K rows g and g + 8, pieces t, t + 4, ..; of V rows 2t, 2t + 1, 2t + 8,
    // 2t + 9, pieces g, g + 8
    uint4 kr[2][KC], vr[4][VC], qr[NT][KC];
    const uint4 zero = make_uint4(0, 0, 0, 0);
    // a step to load: its keys' number in all, key/value head, index, page, and whether it is one of the cache's
    struct Step {
        int n, kvh, s, page;
        bool ok;
    };
    auto page_of = [&](const Segment &z, int s) { return s < z.step1 ? __ldg(z.bt + (s >> 2)) : 0; };
    auto step_of = [&](int n, int kvh, int s, int page, bool any) {
        const bool ok = page >= 0 && page < a.num_pages;
        if (any && !ok) flag(a.status, TS_STATUS_INDEX);
        return Step{n, kvh, s, page, any && ok};
    };
    auto rows_at = [&](const Step &u) { return ((size_t)u.page * a.Hkv + u.kvh) * TS_PAGE_KEYS + (u.s & 3) * 16; };
    auto load_k = [&](const Step &u) {
        const uint4 *p = a.k + rows_at(u) * VEC + t;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int i = 0; i < KC; ++i)
                kr[r][i] = ld_stream(p + (g + 8 * r) * VEC + 4 * i, u.ok && u.s * 16 + g + 8 * r < u.n);
    };
    auto load_v = [&](const Step &u) {
        const uint4 *p = a.v + rows_at(u) * VEC + g;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 2 * t + (r & 1) + 8 * (r >> 1);
#pragma unroll
            for (int i = 0; i < VC; ++i) vr[r][i] = ld_stream(p + row * VEC + 8 * i, u.ok && u.s * 16 + row < u.n);
        }
    };
    auto load_q = [&](const Segment &z) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int h = z.h0 + 8 * j + g;
            const uint4 *p = a.q + z.b * a.q_stride + (size_t)(z.kvh * a.G + h) * VEC + t;
#pragma unroll
            for (int i = 0; i < KC; ++i) qr[j][i] = h < a.G ? __ldg(p + 4 * i) : zero;
        }
    };
    // Four dims of a head, from dd on: where they are final into out, else into a part, with the head's maximum and sum.
    auto put = [&](int b, int kvh, int h0, int h, int dd, const float4 &acc, float top, float sum, float *part) {
        if (part) {
            *reinterpret_cast<float4 *>(part + h * D + dd) = acc;
            if (dd == 0) part[HB * D + h] = top, part[HB * (D + 1) + h] = sum;
        } else {
            const float f = 1.f / sum;
            const __nv_bfloat162 r0 = __floats2bfloat162_rn(acc.x * f, acc.y * f), r1 = __floats2bfloat162_rn(acc.z * f, acc.w * f);
            *reinterpret_cast<uint2 *>(a.out + ((size_t)b * a.Hq + kvh * a.G + h0 + h) * D + dd) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&r0), *reinterpret_cast<const uint32_t *>(&r1));
        }
    };
    // The warps' O, maxima and sums in shared memory as one: the item's rows of out, or a part.
    auto join_warps = [&](int b, int kvh, int h0, float *part) {
        __syncthreads();
        for (int q = tid; q < HB * D / 4; q += kThreads) {
            const int h = q / (D / 4), dd = q % (D / 4) * 4;
            if (h0 + h >= a.G) break;
            float top = -INFINITY, sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w) top = fmaxf(top, m_s[w][h]);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = ex2(m_s[w][h] - guarded(top));
                const float4 y = *reinterpret_cast<const float4 *>(&o_s[w][h][dd]);
                sum = fmaf(l_s[w][h], f, sum);
                acc.x = fmaf(y.x, f, acc.x), acc.y = fmaf(y.y, f, acc.y), acc.z = fmaf(y.z, f, acc.z), acc.w = fmaf(y.w, f, acc.w);
            }
            put(b, kvh, h0, h, dd, acc, top, sum, part);
        }
        __syncthreads();
    };

    // An item in several CTAs' stretches leaves a part of each in the workspace, and the CTA that counts itself last joins
    // them. Many parts are joined in groups of kGroup first, each by its last CTA, which leaves the sum in its first part's
    // place; the last group takes what is left over, so that no group has one part only (whose counter another item could
    // use).
    auto shared_of = [&](const Segment &w) {
        Shared sh{w.b, w.kvh, w.h0};
        if (part_s[1]) {   // (the same thread's)
            sh.c0 = part_s[0], sh.n = part_s[1];
        } else {
            sh.c0 = (int)(((long long)(w.i0 + 1) * ctas - 1) / T);
            sh.n = (int)(((long long)w.i1 * ctas - 1) / T) - sh.c0 + 1;
        }
        sh.k0 = sh.c0;
        sh.groups = sh.n >= kGroupFrom ? sh.n / kGroup : 0;
        if (sh.groups) {
            const int at = min((c - sh.c0) / kGroup, sh.groups - 1);
            sh.k0 = sh.c0 + at * kGroup;
            sh.n = at == sh.groups - 1 ? sh.n - at * kGroup : kGroup;
        }
        return sh;
    };
    Segment z = segment(x);
    bool is_shared[2] = {false, false};
    unsigned counted[2] = {0, 0};
    load_q(z);
    // steps go round the warps, on from segment to segment: turn is the warp that a segment starts with
    int turn = 0;
    auto first_step = [&](const Segment &w) { return w.step0 + warp - turn + (warp < turn ? W : 0); };
    int s = first_step(z), page;           // page: of the step after the one whose loads are under way
    if (s < z.step1) {
        const Step u = step_of(z.n, z.kvh, s, page_of(z, s), true);
        page = page_of(z, s + W);
        load_k(u);
        load_v(u);
    }
    while (true) {
        const bool starts = x == z.i0, ends = z.x1 == z.i1;
        if (!(starts && ends)) {
            is_shared[starts] = true;
            if (tid == 0) shared_s[starts] = shared_of(z);
        }
        // the next segment's first step follows this one's last in the warp's loads
        const bool more = z.x1 < x_end;
        Segment nx;
        int s_nx = 0, page_nx = 0, n_nx = 0, kvh_nx = 0;
        bool step_nx = false;
        if (more) {
            nx = segment(z.x1);
            n_nx = nx.n, kvh_nx = nx.kvh;
            turn = (turn + z.step1 - z.step0) % W;
            s_nx = first_step(nx);
            step_nx = s_nx < nx.step1;
            page_nx = page_of(nx, s_nx);
        }
        if (s >= z.step1 && step_nx) {     // none of this segment's steps is this warp's
            const Step u = step_of(nx.n, nx.kvh, s_nx, page_nx, true);
            page = page_of(nx, s_nx + W);
            load_k(u);
            load_v(u);
        }
        float o[NT][VEC / 2][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            m[j][0] = m[j][1] = -INFINITY;
            l[j][0] = l[j][1] = 0.f;
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
        }
        for (; s < z.step1; s += W) {
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
            const int next = s + W;
            const bool here = next < z.step1;
            const Step u = step_of(here ? z.n : n_nx, here ? z.kvh : kvh_nx, here ? next : s_nx, here ? page : page_nx, here || step_nx);
            load_k(u);
            if (here) page = page_of(z, next + W);
            else if (step_nx) page = page_of(nx, s_nx + W);
            // scores as exponents of 2; keys behind the last one have none
            bool raise = false;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[j][e] = s * 16 + g + 8 * (e >> 1) < z.n ? p[j][e] * a.scale_log2 : -INFINITY;
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
            // (in all 16 bits of each weight). Where nothing is left it counts as 2^-24 of the weight (2^-133 at least, the lowest
            // number there is), so that an infinite value comes through as one; a weight of 0 has neither half
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
                    auto left = [](float w, uint32_t u) {
                        return fminf(w, fmaxf(w - __uint_as_float(u & 0xffff0000u), fmaxf(w * 0x1p-24f, 0x1p-133f)));
                    };
                    const __nv_bfloat162 rest = __floats2bfloat162_rn(left(p0, u0), left(p1, u1));
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
            load_v(u);
        }
        if (more) load_q(nx);

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
        join_warps(z.b, z.kvh, z.h0, starts && ends ? nullptr : a.parts + (size_t)(2 * c + starts) * PART);
        if (!(starts && ends) && tid == 0) counted[starts] = count_up(a.counters + shared_s[starts].k0);
        if (!more) break;
        x = z.x1, z = nx, s = s_nx;
    }

    // ---- parts joined by the CTA that has counted itself last
    for (int side = 0; side < 2; ++side) {
        if (!is_shared[side]) continue;
        const Shared sh = shared_s[side];
        auto last_of = [&](unsigned *counter, unsigned count, unsigned n) {
            if (tid == 0) {
                last_s = count == n - 1;
                if (last_s) *counter = 0, sees_counted();
            }
            __syncthreads();
            const bool yes = last_s;
            __syncthreads();
            return yes;
        };
        // n parts from k0 on, step apart, a warp every W-th; their weights by a warp a head, the first parts' loads under way
        auto join_parts = [&](int k0, int n, int step, float *part) {
            constexpr int NV = HB * D / 128;   // 16-byte pieces of a part a lane
            auto part_at = [&](int i) {
                const int k = k0 + i * step;
                return a.parts + (size_t)(2 * k + (k == sh.c0)) * PART;
            };
            // Few parts: a thread reads its dims of all of them at once (8 requests of 2048 keys, 7 parts: 16.8 us, and 17.8 by
            // warps and shared memory as below).
            if (n <= kFewParts) {
                for (int q = tid; q < HB * D / 4; q += kThreads) {
                    const int h = q / (D / 4), dd = q % (D / 4) * 4;
                    if (sh.h0 + h >= a.G) break;
                    float4 y[kFewParts], sum_y = make_float4(0.f, 0.f, 0.f, 0.f);
                    float mk[kFewParts], lk[kFewParts], top = -INFINITY, sum = 0.f;
#pragma unroll
                    for (int k = 0; k < kFewParts; ++k) {
                        const float *p = part_at(min(k, n - 1));
                        y[k] = __ldcg(reinterpret_cast<const float4 *>(p + h * D + dd));
                        mk[k] = __ldcg(p + HB * D + h), lk[k] = __ldcg(p + HB * (D + 1) + h);
                    }
#pragma unroll
                    for (int k = 0; k < kFewParts; ++k) top = fmaxf(top, mk[k]);
#pragma unroll
                    for (int k = 0; k < kFewParts; ++k)
                        if (k < n) {
                            const float f = ex2(mk[k] - guarded(top));
                            sum = fmaf(lk[k], f, sum);
                            sum_y.x = fmaf(y[k].x, f, sum_y.x), sum_y.y = fmaf(y[k].y, f, sum_y.y);
                            sum_y.z = fmaf(y[k].z, f, sum_y.z), sum_y.w = fmaf(y[k].w, f, sum_y.w);
                        }
                    put(sh.b, sh.kvh, sh.h0, h, dd, sum_y, top, sum, part);
                }
                __syncthreads();
                return;
            }
            float4 acc[NV], v[NV];
            auto load = [&](int k) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int q = i * 32 + lane;
                    acc[i] = make_float4(0.f, 0.f, 0.f, 0.f), v[i] = acc[i];
                    if (k < n && sh.h0 + q / (D / 4) < a.G) v[i] = __ldcg(reinterpret_cast<const float4 *>(part_at(k)) + q);
                }
            };
            load(warp);
            for (int h = warp; h < HB; h += W) {
                constexpr int PL = kMostParts / 32;
                float mk[PL], lk[PL], top = -INFINITY, sum = 0.f;
#pragma unroll
                for (int i = 0; i < PL; ++i) {
                    const int k = lane + 32 * i;
                    const bool in = k < n && sh.h0 + h < a.G;
                    const float *y = part_at(k) + HB * D + h;
                    mk[i] = in ? __ldcg(y) : -INFINITY;
                    lk[i] = in ? __ldcg(y + HB) : 0.f;
                    top = fmaxf(top, mk[i]);
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
#pragma unroll
                for (int i = 0; i < PL; ++i) {
                    const float f = ex2(mk[i] - guarded(top));
                    sum = fmaf(lk[i], f, sum);
                    if (lane + 32 * i < n) f_s[lane + 32 * i][h] = f;
                }
#pragma unroll
                for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                if (lane < W) m_s[lane][h] = top, l_s[lane][h] = lane ? 0.f : sum;
            }
            __syncthreads();
            for (int k = warp; k < n; k += W) {
                float4 now[NV];
#pragma unroll
                for (int i = 0; i < NV; ++i) now[i] = v[i];
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int q = i * 32 + lane;
                    if (k + W < n && sh.h0 + q / (D / 4) < a.G) v[i] = __ldcg(reinterpret_cast<const float4 *>(part_at(k + W)) + q);
                }
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const float f = f_s[k][(i * 32 + lane) / (D / 4)];
                    acc[i].x = fmaf(now[i].x, f, acc[i].x), acc[i].y = fmaf(now[i].y, f, acc[i].y);
                    acc[i].z = fmaf(now[i].z, f, acc[i].z), acc[i].w = fmaf(now[i].w, f, acc[i].w);
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int q = i * 32 + lane;
                *reinterpret_cast<float4 *>(&o_s[warp][q / (D / 4)][q % (D / 4) * 4]) = acc[i];
            }
            join_warps(sh.b, sh.kvh, sh.h0, part);
        };
        if (!last_of(a.counters + sh.k0, counted[side], sh.n)) continue;
        if (!sh.groups) {
            join_parts(sh.c0, sh.n, 1, nullptr);
            continue;
        }
        join_parts(sh.k0, sh.n, 1, a.parts + (size_t)(2 * sh.k0 + (sh.k0 == sh.c0)) * PART);
        unsigned *const over = a.counters + gridDim.x + sh.c0;
        unsigned count = 0;
        if (tid == 0) count = count_up(over);
        if (last_of(over, count, sh.groups)) join_parts(sh.c0, sh.groups, kGroup, nullptr);
    }
}

template <int D, int NT, bool ONE>
int grid_of() {
    return std::min(kMostCtas, num_sms() * kPerSm<D, NT, ONE>);
}
int most_ctas(int d, int HB) {
    return d == 64 ? (HB == 8 ? grid_of<64, 1, false>() : grid_of<64, 2, false>())
                   : (HB == 8 ? grid_of<128, 1, false>() : grid_of<128, 2, false>());
}
int heads_of(int G) { return G > 8 ? 16 : 8; }
size_t counter_bytes() { return (size_t)(kMostCtas + 1) * 8; }   // any grid's

template <int D, int NT, bool ONE>
cudaError_t launch_as(const DecodeArgs &a, cudaStream_t s) {
    constexpr auto kern = k_attn_decode<D, NT, ONE>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D, NT, ONE>);
    if (e != cudaSuccess) return e;
    return launch(kern, dim3(grid_of<D, NT, ONE>()), dim3(32 * kWarps<D, NT, ONE>), kSmem<D, NT, ONE>, s, a);
}
template <int D, int NT>
cudaError_t launch_decode(const DecodeArgs &a, cudaStream_t s) {
    return (long long)a.B * a.Hkv * a.blocks <= kFewItems ? launch_as<D, NT, true>(a, s) : launch_as<D, NT, false>(a, s);
}

}  // namespace

// Counters first: one workspace serves calls of several sizes.
size_t decode_ws_bytes(int B, int Hq, int Hkv, int d) {
    const int HB = heads_of(Hq / Hkv);
    return counter_bytes() + (size_t)most_ctas(d, HB) * 2 * HB * (d + 2) * 4;
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
    if (d == 128) return HB == 8 ? launch_decode<128, 1>(a, s) : launch_decode<128, 2>(a, s);
    return HB == 8 ? launch_decode<64, 1>(a, s) : launch_decode<64, 2>(a, s);
}

}  // namespace ts
