// sample.cu -- a token a row from logits and a uniform number: temperature,
// top-k, top-p and min-p.
//
// Order of a row's tokens: value falling, id rising. What is kept is a start of
// that order, so it is given by the value of its last token and by how many of
// the tokens of that value are kept (the lowest ids). The three filters only
// shorten it.
//
// Whether a token is kept, and which token a uniform number falls on, are
// comparisons of sums over a vocabulary: in fp32 a row of 50k tokens is decided
// wrongly about once in a thousand draws. So sums are whole numbers, whose order
// does not matter, of weights that are right to 2^-23.2 of themselves (Weights), and
// so off by a bound that is known. Where u or top_p falls within that bound of a
// border (one row of 50k tokens in some four hundred), it is weighed once more, to
// 2^-43 (exact_sum), and decided by that: as in 64-bit floating point, but for what
// that itself leaves open.
//
// Passes over a row: maximum; where a filter needs it a bound of the candidates
// for the last token kept, and these; kept weights; output rows. Three layouts:
//  kCluster  a cluster of CTAs a row, each a segment in shared memory: the row is
//            read once, the passes cost instructions (some twenty an element)
//  kStream   a CTA a row, read again from L2, for many filtered long rows: none of
//            a cluster's barriers, and room for thousands of candidates
//  kSmall    a small CTA a row, for many short rows
// One row is a chain of latencies (32000 bf16, top-k and top-p: 10.2 us, of which
// launch and row 4, the cluster's barriers 4); 64 rows of 50272 drawn from the whole
// distribution 10.9 us; 1024 filtered rows with their distributions 137 us, 44% of
// the copy rate: the passes' latencies, and issue slots. A row of 50272 that is
// weighed once more takes 8 (alone) to 19 us (with 63 others) for it.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "attn_common.cuh"
#include "decode.cuh"

namespace ts {
namespace {

namespace cg = cooperative_groups;

typedef unsigned long long u64;
enum Mode { kCluster, kStream, kSmall };
template <Mode M>
struct Cfg {
    static constexpr int NT = M == kSmall ? 128 : 512, W = NT / 32;
    static constexpr int BINS = M == kSmall ? 256 : 512;
    static constexpr int LIST = M == kStream ? 6144 : 512, SORT = M == kStream ? 4096 : 512;   // candidates, and how many can be sorted
    static constexpr int REP = M == kStream ? 4 : 1;         // histograms, so that none counts more than 2^16 + 2^10 elements
    static constexpr int PER_SM = M == kSmall ? 8 : 2;       // CTAs
};
constexpr int kGroup = 128;       // elements of a warp's turn
// Up to so many rows are taken in an order of their settings (in order and not: settings by row and distributions, 1024 rows of
// 50272 139 us and 158, 2048 rows 253 and 261; all with top-k 50 80 and 76, 145 and 137).
constexpr int kOrderedRows = 2048;
constexpr int kRing = 4;           // groups of a warp in shared memory or on their way there, where rows are read again

// Whole numbers in the order of the floats (-0 counts as 0).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// A number from [0, 1) in units of 2^-64.
__device__ __forceinline__ u64 part64(float x) { return __float2ull_rz(x * 18446744073709551616.f); }

// A token's place in the order as one rising number.
constexpr int kIdBits = 18;
__device__ __forceinline__ u64 order_of(uint32_t key, int id) { return (u64)(uint32_t)~key << kIdBits | (uint32_t)id; }

// 2^(j / 32) in units of 2^-62.
__device__ const u64 kRoot[32] = {
    0x4000000000000000ull, 0x4166c34c5615d0ecull, 0x42d561b3e6243d8aull, 0x444c0740496d4294ull, 0x45cae0f1f545eb73ull,
    0x47521cc5a2e6a9e0ull, 0x48e1e9b9d588e19bull, 0x4a7a77d47f7b84b1ull, 0x4c1bf828c6dc54b8ull, 0x4dc69cdceaa72a9cull,
    0x4f7a993048d088d7ull, 0x513821818624b40cull, 0x52ff6b54d8a89c75ull, 0x54d0ad5a753e077cull, 0x56ac1f752150a563ull,
    0x5891fac0e95612c8ull, 0x5a827999fcef3242ull, 0x5c7dd7a3b17dcf75ull, 0x5e8451cfac061b5full, 0x6096266533384a2bull,
    0x62b39508aa836d6full, 0x64dcdec3371793d1ull, 0x6712460a8fc24072ull, 0x69540ec8f895722dull, 0x6ba27e656b4eb57aull,
    0x6dfddbcbed791babull, 0x70666f76154a7089ull, 0x72dc8373be41a454ull, 0x75606373ee921c97ull, 0x77f25ccdee6d7ae6ull,
    0x7a92be8a92436616ull, 0x7d41d96db915019dull};

// Two floats in one register pair, worked on at once.
__device__ __forceinline__ u64 two(float a, float b) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void one_each(u64 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ u64 shifted(u64 v, int by) {   // 0 from 64 on
    u64 r;
    asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(v), "r"(by));
    return r;
}

// exp((x - top) / T) = 2^y to some 2^-43 of itself (near the top 2^-44), in units of 2^(drop - 62). y = (x - top) c,
// c = log2(e) / T = ch + cl; by of x and top: 1, or 2^-64 where T is above 2^100, so that no difference that counts overflows.
// The difference and the products with their errors: y = Y - r, Y = n + j / 32 + g; t = (g - r) ln 2 and its square as sums of two
// floats, 2^(g - r) = 1 + t + t^2 / 2 + .. in whole numbers of 2^-62 where it is large. (-inf: 0)
__device__ __forceinline__ u64 exact_of(float x, float top, float ch, float cl, float by, int drop) {
    const float v = __fmul_rn(x, -by), d = __fadd_rn(v, top), b = __fsub_rn(d, v);
    const float low = __fadd_rn(__fsub_rn(v, __fsub_rn(d, b)), __fsub_rn(top, b));   // d + low = top - x
    const float Y = __fmul_rn(d, -ch), r = __fmaf_rn(low, ch, __fmaf_rn(d, cl, __fmaf_rn(d, ch, Y)));
    const int m = __float2int_rn(fmaxf(Y, -100.f) * 32.f);
    const float g = __fmaf_rn((float)m, -0.03125f, Y);
    const float L = 0.693147182464599609375f, Ll = -1.904654299957767e-09f;   // ln 2
    const float t = __fmul_rn(g, L), tl = __fmaf_rn(r, -L, __fmaf_rn(g, Ll, __fmaf_rn(g, L, -t)));
    const float q = __fmul_rn(t, t), ql = __fmaf_rn(tl, tl, __fmaf_rn(t, 2.f * tl, __fmaf_rn(t, t, -q)));
    const float rest = tl + fmaf(0.5f, ql, fmaf(q * 0.5f, fmaf(t * (1.f / 3), tl, tl), t * q * fmaf(t, fmaf(t, 1.f / 120, 1.f / 24), 1.f / 6)));
    // (conversions to 64 bits are several times slower than these four)
    const int t31 = __float2int_rn(t * 0x1p31f);
    const long long p = ((long long)t31 << 31) + __float2int_rn(__fmaf_rn((float)t31, -0x1p-31f, t) * 0x1p62f) +
                        ((long long)__float2int_rn(q * 0x1p43f) << 18) + ((long long)__float2int_rn(rest * 0x1p47f) << 15);
    const u64 R = kRoot[m & 31];
    return Y > -100.f ? shifted(R + (u64)__mul64hi((long long)R, p << 2), drop - (m >> 5)) : 0;
}
// (not inlined: for rows that are weighed once more, and the tokens at their borders)
__device__ __noinline__ u64 exact_one(float x, float top, float ch, float cl, float by, int drop) {
    return exact_of(x, top, ch, cl, by, drop);
}
__device__ __noinline__ u64 exact_sum(float x0, float x1, float x2, float x3, float top, float ch, float cl, float by, int drop) {
    return exact_of(x0, top, ch, cl, by, drop) + exact_of(x1, top, ch, cl, by, drop) + exact_of(x2, top, ch, cl, by, drop) +
           exact_of(x3, top, ch, cl, by, drop);
}

// 2^(x c - N), c = log2(e) / T = ch + cl and N the whole number next to top c: the weights of all tokens times one number from
// [0.7, 1.42], which no comparison of their sums sees. x c = n + f, n whole and |f| <= 1/2 (the difference of x ch and n is rounded
// once, whatever they are), 2^f by a polynomial (interpolated at Chebyshev's points, 2^-26.7 of itself), n in the exponent. Off by
// at most: the polynomial and its roundings 2^-23.69 (at every fp32 number), the two roundings of f 2^-25.5, c - ch - cl 2^-28 (at
// |x c| = 2^22): kOff. Then as whole numbers of 2^-42, the nearest. Where top c is above that limit, x and top are their distances
// from top before, exact where they are less than 100 / c; where T is above 2^100, both are times `by` before.
constexpr float kUnits = 4398046511104.f;    // 2^42
constexpr int kUnitBits = 42;
constexpr float kOff = 0x1.bp-24f;
constexpr float kMagic = 12582912.f;         // 1.5 * 2^23: a sum with it is a whole number in its lower bits
// Numbers from [0, 2) as a 2^-20 + b 2^-42, a and b whole, |b| <= 2^21, in the lower bits of sums with these:
constexpr float kHigh = 0x1.8p3f, kLow = 0x1.8p-19f;
constexpr uint32_t kHighBits = 0x41400000u, kLowBits = 0x36400000u;
struct Weights {
    float top, ch, cl, by;   // (top times by: for exact weights, and distributions)
    float floor, magic;      // what is below the former weighs as that, less than a unit; kMagic - N
    float pivot;             // x counts as x by - pivot
    // (x - top) c, rounded; falls with x, or stays
    __device__ __forceinline__ float exponent(float x) const { return __fmul_rn(__fadd_rn(__fmul_rn(x, -by), top), -ch); }
    __device__ __forceinline__ u64 exact(float x0, float x1, float x2, float x3, int drop) const {
        return exact_sum(x0, x1, x2, x3, top, ch, cl, by, drop);
    }
    __device__ __forceinline__ u64 exact(float x, int drop) const { return exact_one(x, top, ch, cl, by, drop); }
    __device__ __forceinline__ void four(const float (&x)[4], float (&w)[4]) const {
        const u64 h = two(ch, ch), l = two(cl, cl), minus = two(-1.f, -1.f), c = two(magic, magic);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            float y0, y1;
            one_each(fma2(two(x[e], x[e + 1]), two(by, by), two(-pivot, -pivot)), y0, y1);
            const u64 v = two(fmaxf(y0, floor), fmaxf(y1, floor)), k = fma2(v, h, c);
            const u64 f = fma2(v, l, fma2(v, h, fma2(k, minus, c)));
            u64 q = fma2(f, two(0x1.4413dcp-13f, 0x1.4413dcp-13f), two(0x1.5f0906p-10f, 0x1.5f0906p-10f));
            q = fma2(f, q, two(0x1.3b2a52p-7f, 0x1.3b2a52p-7f));
            q = fma2(f, q, two(0x1.c6af6cp-5f, 0x1.c6af6cp-5f));
            q = fma2(f, q, two(0x1.ebfbe0p-3f, 0x1.ebfbe0p-3f));
            q = fma2(f, q, two(0x1.62e430p-1f, 0x1.62e430p-1f));
            float k0, k1, p0, p1;
            one_each(k, k0, k1);
            one_each(fma2(f, q, two(1.f, 1.f)), p0, p1);
            w[e] = __int_as_float(__float_as_int(p0) + (int)((uint32_t)__float_as_int(k0) << 23));   // (kMagic's bits are above 2^9)
            w[e + 1] = __int_as_float(__float_as_int(p1) + (int)((uint32_t)__float_as_int(k1) << 23));
        }
    }
    __device__ __forceinline__ static u64 whole(float w) {
        const float a = __fadd_rn(w, kHigh), b = __fadd_rn(__fsub_rn(w, __fsub_rn(a, kHigh)), kLow);
        return ((u64)(__float_as_uint(a) - kHighBits) << 22) + (long long)(int)(__float_as_uint(b) - kLowBits);
    }
    // (not inlined: it is for few)
    __device__ __noinline__ static u64 one(float x, float ch, float cl, float floor, float magic) {
        x = fmaxf(x, floor);
        const float k = __fmaf_rn(x, ch, magic), f = __fmaf_rn(x, cl, __fmaf_rn(x, ch, __fsub_rn(magic, k)));
        float q = __fmaf_rn(f, 0x1.4413dcp-13f, 0x1.5f0906p-10f);
        q = __fmaf_rn(f, q, 0x1.3b2a52p-7f);
        q = __fmaf_rn(f, q, 0x1.c6af6cp-5f);
        q = __fmaf_rn(f, q, 0x1.ebfbe0p-3f);
        q = __fmaf_rn(f, __fmaf_rn(f, q, 0x1.62e430p-1f), 1.f);
        return whole(__int_as_float(__float_as_int(q) + (int)((uint32_t)__float_as_int(k) << 23)));
    }
    __device__ __forceinline__ u64 operator()(float x) const {
        return one(__fmaf_rn(x, by, -pivot), ch, cl, floor, magic);
    }
    // Weights as floats, the largest `one`, to some 2^-21 of themselves.
    __device__ __forceinline__ float real(float x, float one) const {
        x *= by;
        const float dh = x - top, bb = dh - x, dl = (x - (dh - bb)) - (top + bb), yh = dh * ch;
        const float yl = fmaf(dh, ch, -yh) + fmaf(dh, cl, dl * ch);
        return yh > -150.f ? ex2(yh) * fmaf(yl, 0.693147182f, 1.f) * one : 0.f;
    }
    __device__ __forceinline__ void real4(const float (&x)[4], float one, float (&p)[4]) const {
        const u64 b = two(by, by), t = two(-top, -top), h = two(ch, ch), l = two(cl, cl), minus = two(-1.f, -1.f);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const u64 v = mul2(two(x[e], x[e + 1]), b), d = add2(v, t), bb = fma2(v, minus, d),
                      low = add2(fma2(fma2(bb, minus, d), minus, v), fma2(bb, minus, t));   // d + low = x - top
            const u64 y = mul2(d, h), yl = add2(fma2(d, h, mul2(y, minus)), fma2(d, l, mul2(low, h)));
            float y0, y1, f0, f1;
            one_each(y, y0, y1);
            one_each(fma2(yl, two(0.693147182f, 0.693147182f), two(1.f, 1.f)), f0, f1);
            p[e] = y0 > -150.f ? ex2(y0) * f0 * one : 0.f, p[e + 1] = y1 > -150.f ? ex2(y1) * f1 * one : 0.f;
        }
    }
};

// The sum of weights as whole numbers, below 2^10 of them, in two 32-bit sums.
struct WeightSum {
    uint32_t a = 0, b = 0;
    __device__ __forceinline__ void add(const float (&w)[4]) {
        const u64 high = two(kHigh, kHigh), minus = two(-kHigh, -kHigh), low = two(kLow, kLow);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
            const u64 v = two(w[e], w[e + 1]), s = add2(v, high);
            const u64 t = add2(fma2(add2(s, minus), two(-1.f, -1.f), v), low);
            float s0, s1, t0, t1;
            one_each(s, s0, s1);
            one_each(t, t0, t1);
            a += __float_as_uint(s0) + __float_as_uint(s1) - 2 * kHighBits;
            b += __float_as_uint(t0) + __float_as_uint(t1) - 2 * kLowBits;
        }
    }
    __device__ __forceinline__ u64 sum() const { return ((u64)a << 22) + (long long)(int)b; }
    __device__ __forceinline__ u64 warp_sum() const {   // of four each
        return ((u64)__reduce_add_sync(~0u, a) << 22) + (long long)__reduce_add_sync(~0u, (int)b);
    }
};

// Four elements of a row as floats.
__device__ __forceinline__ void load4(const float *p, float (&x)[4]) {
    const float4 v = *reinterpret_cast<const float4 *>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4]) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}
// An atomic sum in shared memory by halves, as there is no 64-bit one but by comparing and trying again.
__device__ __forceinline__ void add64(u64 *p, u64 v) {
    uint32_t *const q = reinterpret_cast<uint32_t *>(p);
    const uint32_t lo = (uint32_t)v, hi = (uint32_t)(v >> 32) + (atomicAdd(q, lo) + lo < lo);
    if (hi) atomicAdd(q + 1, hi);
}
__device__ __forceinline__ u64 warp_scan(u64 v) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(~0u, v, o);
        if ((threadIdx.x & 31) >= o) v += y;
    }
    return v;
}

template <Mode M>
struct Shared {
    using F = Cfg<M>;
    uint32_t h[F::REP][3][F::BINS];   // the segment's histogram: counts in [0], or sums by 15, 15 and the rest of the bits
    u64 list[F::LIST];                // the cluster's candidates, in its first CTA, by their place in the order
    union {
        u64 part[F::W];
        float top[F::W];
    };
    u64 from[2][8];                   // what the cluster's CTAs tell one another, in turn
    u64 cut, kept;                    // the last token kept, the sum of all kept weights
    u64 most;                         // the last one that top-k alone leaves
    u64 above, total;
    uint4 ring[M == kStream ? F::W * kRing * 32 : 1];   // groups on their way, the warps' own
    float ch, cl, mh, ml;             // log2(e) / T and T ln(min_p), as sums of two floats
    int n_list, n_kept, at;
    bool cut_unsure, draw_unsure;     // by less than the sums may be off
};
static_assert(sizeof(Shared<kCluster>) <= 10752, "two CTAs an SM with 25216 fp32 elements each");
template <Mode M>
constexpr size_t kFixed = (sizeof(Shared<M>) + 15) / 16 * 16;   // then a sum a unit, then the segment

__device__ __forceinline__ void copy16(void *to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}

// A cluster a row, segment SL elements; but for kCluster a CTA a row, its segment the row. Positions count from the 16-byte
// boundary at or before the row's first element (lead elements before it); those outside the row count as -inf.
template <typename T, Mode M>
__global__ void __launch_bounds__(Cfg<M>::NT, Cfg<M>::PER_SM) k_sample(SampleArgs a, int SL) {
    extern __shared__ uint4 smem[];
    using F = Cfg<M>;
    using Sh = Shared<M>;
    constexpr int NT = F::NT, W = F::W, BINS = F::BINS, LIST = F::LIST, SORT = F::SORT;
    constexpr bool STREAM = M == kStream, ONE = M != kCluster;
    Sh &sm = *reinterpret_cast<Sh *>(smem);
    const int NG = SL / kGroup;
    u64 *const sums = reinterpret_cast<u64 *>(reinterpret_cast<char *>(smem) + kFixed<M>);   // kept weights of each unit
    T *const seg = reinterpret_cast<T *>(sums + (STREAM ? (NG + 1) / 2 * 2 : NT));
    const cg::cluster_group cluster = cg::this_cluster();
    const int C = ONE ? 1 : cluster.num_blocks(), rank = ONE ? 0 : cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.V;
    int r = blockIdx.x / C;
    auto sync = [&] {
        if (ONE || C == 1) __syncthreads();
        else cluster.sync();
    };
    auto peer = [&](int c) -> Sh & {
        if constexpr (ONE) return sm;
        else return *cluster.map_shared_rank(&sm, c);
    };
    if (!ONE && C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // the cluster's CTAs are there:
    pdl_wait();
    pdl_trigger();
    // Rows of unlike settings are taken the long ones first, so that none of these is all that is left at the end: top-p alone,
    // then nothing or a large k, then the others. Every CTA counts for itself which is its.
    if constexpr (STREAM)
        if (a.R <= kOrderedRows && a.top_p && (a.top_k || a.min_p)) {
            constexpr int Q = kOrderedRows / NT;
            u64 mine = 0;
            int kind[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int i = tid * Q + q;
                kind[q] = -1;
                if (i >= a.R) continue;
                const int k = a.top_k ? a.top_k[i] : 0;
                const bool few = (a.min_p && a.min_p[i] > 0.f) || (k > 0 && k <= NT) || (a.temperature && a.temperature[i] == 0.f);
                kind[q] = few ? 2 : (k > 0 && k < V) || a.top_p[i] >= 1.f;
                mine += 1ull << 20 * kind[q];
            }
            u64 upto = warp_scan(mine);
            if (lane == 31) sm.part[warp] = upto;
            __syncthreads();
            u64 all = 0;
            for (int w = 0; w < W; ++w) {
                if (w < warp) upto += sm.part[w];
                all += sm.part[w];
            }
            constexpr int ONES = (1 << 20) - 1;
            const int n0 = (int)(all & ONES), n1 = (int)(all >> 20 & ONES), which = r < n0 ? 0 : r < n0 + n1 ? 1 : 2;
            int at = (int)(upto - mine >> 20 * which & ONES) + (which == 0 ? 0 : which == 1 ? n0 : n0 + n1);
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (kind[q] == which && at++ == r) sm.at = tid * Q + q;
            __syncthreads();
            r = sm.at;
            __syncthreads();
        }

    const T *const row = reinterpret_cast<const T *>(a.logits) + (size_t)r * a.stride;
    const int lead = (int)(((uintptr_t)row & 15) / sizeof(T)), base = rank * SL;
    constexpr int VE = 16 / sizeof(T);
    // 16-byte pieces that lie within the row; what is left at the segment's ends, one by one
    const int v_lo = min(SL, max(0, lead - base + VE - 1)) / VE, v_hi = max(v_lo, min(SL, max(0, V + lead - base)) / VE);
    const uint4 *const pieces = reinterpret_cast<const uint4 *>(row - lead) + base / VE;
    if constexpr (!STREAM)
        for (int v = v_lo + tid; v < v_hi; v += NT) copy16(seg + v * VE, pieces + v);
    const float temp = a.temperature ? a.temperature[r] : 1.f, top_p = a.top_p ? a.top_p[r] : 1.f,
                min_p = a.min_p ? a.min_p[r] : 0.f, u = a.u ? a.u[r] : 0.f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    const bool wrong =
        !(temp >= 0.f && temp < INFINITY) || isnan(top_p) || isnan(min_p) || top_k < 0 || !(u >= 0.f && u < 1.f);
    const bool greedy = temp < 7.888609052210118e-31f;   // 2^-100
    const float by = temp > 1.2676506002282294e30f ? 5.421010862427522e-20f : 1.f;   // 2^-64 above 2^100
    if (tid == 0) {   // (64-bit arithmetic is slow enough here that one thread does it for all)
        const double c = 1.4426950408889634 / (greedy ? 1.0 : (double)(temp * by));
        sm.ch = (float)c;
        sm.cl = (float)(c - (double)sm.ch);
        if (min_p > 0.f) {
            const double m = (double)temp * log((double)fminf(min_p, 1.f));
            sm.mh = (float)m, sm.ml = (float)(m - (double)sm.mh);
        }
        sm.n_list = 0;
        sm.draw_unsure = false;
    }
    auto empty = [&] {
        uint32_t *const h = &sm.h[0][0][0];
#pragma unroll
        for (int i = 0; i < F::REP * 3 * BINS; i += NT) h[i + tid] = 0;
    };
    empty();

    // ---- the row's maximum; of each thread's elements four, of every fourth one
    float own[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    bool bad = false;
    auto look = [&](const T *p) {
        float f[4];
        load4(p, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bad |= !(f[e] < INFINITY);
            own[e] = fmaxf(own[e], f[e]);
        }
        return fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));
    };
    const int odd = STREAM ? v_lo * VE + max(0, V + lead - v_hi * VE) : SL - (v_hi - v_lo) * VE;
    for (int i = tid; i < odd; i += NT) {
        const int pos = i < v_lo * VE ? i : i + (v_hi - v_lo) * VE, p = base + pos - lead;
        const T x = p >= 0 && p < V ? row[p] : (T)(-INFINITY);
        if constexpr (!STREAM) seg[pos] = x;
        bad |= !((float)x < INFINITY);
        own[0] = fmaxf(own[0], (float)x);
    }
    // the largest of every 32 pieces (as key_of); the ends of the row, which are not all pieces, count as the largest there is
    uint32_t *const most_of = reinterpret_cast<uint32_t *>(sums);
    constexpr int CG = 32 * VE / kGroup;   // groups that one stands for
    if constexpr (STREAM) {
        const int chunks = (NG + CG - 1) / CG;
        for (int c0 = warp; c0 < chunks; c0 += 4 * W) {
            uint4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int v = (c0 + k * W) * 32 + lane;
                if (v >= v_lo && v < v_hi) x[k] = pieces[v];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int chunk = c0 + k * W, v = chunk * 32 + lane;
                if (chunk >= chunks) break;
                float most = INFINITY;
                if (v >= v_lo && v < v_hi) {
                    most = -INFINITY;
#pragma unroll
                    for (int i = 0; i < VE; i += 4) most = fmaxf(most, look(reinterpret_cast<const T *>(&x[k]) + i));
                }
                const uint32_t key = __reduce_max_sync(~0u, key_of(most));
                if (lane == 0) most_of[chunk] = key;
            }
        }
    } else {
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 2
        for (int v = v_lo + tid; v < v_hi; v += NT)   // the pieces that this thread has copied
#pragma unroll
            for (int i = 0; i < VE; i += 4) look(seg + v * VE + i);
    }
    float top = fmaxf(fmaxf(own[0], own[1]), fmaxf(own[2], own[3]));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) sm.top[warp] = top;
    bad = __syncthreads_or(bad);
    top = sm.top[lane % W];
#pragma unroll
    for (int o = W / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    const float ch = sm.ch;
    // a lower bound of the row's sum of weights: these tokens' (a number, whatever the settings: NaN says that logits are bad)
    float some = 1.f;
    const bool bound = !wrong && top_p < 1.f && (top_k <= 0 || top_k >= V) && !(min_p > 0.f);
    if (bound) {
        some = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) some += own[e] > -INFINITY ? ex2((own[e] - top) * by * ch) : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) some += __shfl_xor_sync(~0u, some, o);
        __syncthreads();
        if (lane == 0) sm.top[warp] = some;
        __syncthreads();
        some = sm.top[lane % W];
#pragma unroll
        for (int o = W / 2; o; o >>= 1) some += __shfl_xor_sync(~0u, some, o);
    }
    // one word to every CTA of the cluster; all of theirs, in the cluster's order
    int turn = 0;
    auto tell = [&](u64 word) {
        u64 *const mine = sm.from[turn];
        if (tid < C) peer(tid).from[turn][rank] = word;
        turn ^= 1;
        sync();
        return mine;
    };
    if (!ONE && C > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // before anything is written to them
    const u64 *const tops = tell((u64)__float_as_uint(top) | (u64)__float_as_uint(bad ? NAN : some) << 32);
    for (int c = 0; c < C; ++c) top = fmaxf(top, __uint_as_float((uint32_t)tops[c]));
    some = 0.f;
    for (int c = 0; c < C; ++c) {
        const float t = __uint_as_float((uint32_t)tops[c]), x = __uint_as_float((uint32_t)(tops[c] >> 32));
        bad |= isnan(x);
        if (t > -INFINITY) some += x * ex2((t - top) * by * ch);
    }
    bad |= top == -INFINITY;

    // four elements of the segment from position pos on, a multiple of 4
    auto get4 = [&](int pos, float (&x)[4]) {
        if constexpr (STREAM) {
            const int p = pos - lead;
            if ((unsigned)p <= (unsigned)(V - 4)) load4(row + p, x);   // (V is large)
            else
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = p + e >= 0 && p + e < V ? (float)row[p + e] : -INFINITY;
        } else {
            load4(seg + pos, x);
        }
    };
    float *const p_to = a.probs ? a.probs + (size_t)r * V : nullptr, *const k_to = a.kept ? a.kept + (size_t)r * V : nullptr;
    auto put4 = [&](float *to, int p, const float (&y)[4]) {   // ids p .. p + 3 of an output row
        if ((((uintptr_t)to - (uintptr_t)lead * 4) & 15) == 0 && p >= 0 && p + 4 <= V)
            __stcs(reinterpret_cast<float4 *>(to + p), make_float4(y[0], y[1], y[2], y[3]));
        else
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (p + e >= 0 && p + e < V) to[p + e] = y[e];
    };
    auto fill_rows = [&](float prob, float logit) {   // the segment's part of them with one number
        for (int k = 0; k < 2; ++k) {
            float *const to = k ? k_to : p_to;
            const float v = k ? logit : prob, y[4] = {v, v, v, v};
            if (to)
                for (int i = tid; i < SL / 4; i += NT) put4(to, base + 4 * i - lead, y);
        }
    };
    if (bad || wrong) {
        if (rank == 0 && tid == 0) {
            flag(a.status, (bad ? TS_STATUS_NONFINITE : 0u) | (wrong ? TS_STATUS_INDEX : 0u));
            if (a.token) a.token[r] = -1;
        }
        fill_rows(NAN, NAN);
        sync();
        return;
    }
    // (4.0e6 is below 2^22: sums with kMagic - N are exact)
    const bool far = !(fabsf(top * by * ch) < 4.0e6f);
    const float pivot = far ? top * by : 0.f, highest = top * by - pivot;
    const Weights weight{top * by, ch, sm.cl, by, highest - 100.f / ch, kMagic - rintf(highest * ch), pivot};
    // tokens below this are not kept: min-p (the sum rounded up), and -inf
    float low = -3.402823466e38f;
    if (min_p > 0.f && !greedy) {
        const float s = top + sm.mh, bb = s - top, e = (top - (s - bb)) + (sm.mh - bb);
        low = fmaxf(low, __fadd_ru(s, e + sm.ml));
    }
    float cut = low;               // kept: above this value, or this value and an id up to cut_id
    int cut_id = 1 << kIdBits;
    auto kept = [&](float x, int id) { return x > cut || (x == cut && id <= cut_id); };
    auto cut_at = [&](u64 last) {
        cut = value_of(~(uint32_t)(last >> kIdBits));
        cut_id = (int)(last & ((1 << kIdBits) - 1));
    };
    auto all_of_them = [](float, int, float) { return true; };
    auto kept_of_them = [&](float v, int i, float) { return kept(v, i); };

    // every element of the segment, by groups: f(group, x[4], id of x[0])
    auto groups = [&](auto f) {
        float x[4], next[4];
        if (warp < NG) get4(warp * kGroup + lane * 4, next);
#pragma unroll 1
        for (int g = warp; g < NG; g += W) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = next[e];
            if (g + W < NG) get4((g + W) * kGroup + lane * 4, next);
            f(g, x, base + g * kGroup + lane * 4 - lead);
        }
    };
    // The same where f is short: what comes from L2 is on its way through shared memory kRing - 1 turns before its use, each
    // lane's part by itself. (1024 rows of 50272, top-k 1000: 158 us and 168; with a longer f that costs registers, top-p 0.95:
    // 270 and 252.)
    auto groups_ahead = [&](auto f) {
        if constexpr (STREAM) {
            constexpr unsigned STAGE = kGroup * sizeof(T), RING = kRing * STAGE;
            const T *const mine = reinterpret_cast<const T *>(sm.ring) + warp * kRing * kGroup + lane * 4;
            const uint32_t ring = smem_u32(mine);
            const unsigned last = V - 4;                              // the last place of four tokens; others are none or fewer
            const T *from = row + (warp * kGroup + lane * 4 - lead);
            unsigned p = warp * kGroup + lane * 4 - lead, p_from = p, stage = 0;
            auto fetch = [&](unsigned to) {
                if (p_from <= last)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(ring + to), "l"(from), "n"(4 * sizeof(T)) : "memory");
                asm volatile("cp.async.commit_group;" ::: "memory");
                from += W * kGroup, p_from += W * kGroup;
            };
#pragma unroll
            for (int k = 0; k < kRing - 1; ++k) fetch(k * STAGE);
            float x[4];
#pragma unroll 1
            for (int g = warp; g < NG; g += W) {
                fetch((stage + (kRing - 1) * STAGE) % RING);         // where the last turn's was
                asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
                if (p <= last) load4(mine + stage / sizeof(T), x);
                else get4(p + lead, x);
                f(g, x, p);
                p += W * kGroup;
                stage = (stage + STAGE) % RING;
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        } else {
            groups(f);
        }
    };
    // The groups that may have a value from `from` on, where the largest ones are known and tell few.
    auto high_groups = [&](float from, auto f) {
        if constexpr (STREAM) {
            const uint32_t key = key_of(from);
            auto high = [&](int j0) {   // of the warp's groups warp + j W those of j0 .. j0 + 31
                const int g = warp + (j0 + lane) * W;
                return __ballot_sync(~0u, g < NG && most_of[g / CG] >= key);
            };
            int n = 0;
            for (int j0 = 0; warp + j0 * W < NG; j0 += 32) n += __popc(high(j0));
            if (2 * n * W <= NG)
                for (int j0 = 0; warp + j0 * W < NG; j0 += 32)
                    for (unsigned m = high(j0); m;) {
                        constexpr int U = 4;   // at once
                        float x[U][4];
                        int g[U];
#pragma unroll
                        for (int q = 0; q < U; ++q) {
                            g[q] = -1;
                            if (!m) continue;
                            g[q] = warp + (j0 + __ffs(m) - 1) * W;
                            m &= m - 1;
                            get4(g[q] * kGroup + lane * 4, x[q]);
                        }
#pragma unroll
                        for (int q = 0; q < U; ++q)
                            if (g[q] >= 0) f(g[q], x[q], g[q] * kGroup + lane * 4 - lead);
                    }
            else groups_ahead(f);
        } else {
            groups(f);
        }
    };
    // Sums of kept weights are held by units: a group of kGroup, or, where the row is in shared memory, a thread's stretch of an
    // odd number of elements (read without conflicts of banks, and its sum needs no other thread's).
    const int unit = STREAM ? kGroup : (SL + NT - 1) / NT | 1, units = STREAM ? NG : NT;
    // four elements of a stretch from position i on
    auto four_at = [&](int i, int end, float (&x)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = i + e < end ? (float)seg[i + e] : -INFINITY;
    };
    // The weights of a thread's stretch, four at a time: add(x[4], w[4], id of x[0]).
    auto weigh_stretch = [&](auto add) {
        const int i0 = min(SL, tid * unit), i1 = min(SL, i0 + unit);
#pragma unroll 1
        for (int i = i0; i < i1; i += 4) {
            float x[4], w[4];
            four_at(i, i1, x);
            weight.four(x, w);
            add(x, w, base + i - lead);
        }
    };
    // The sums of the groups' weights, of the elements that take(value, id, Y) says; see(group, x[4], w[4]) looks at all.
    auto sum_groups_and = [&](auto each, auto see, auto take) {
        each([&](int g, const float (&x)[4], int id) {
            float w[4];
            weight.four(x, w);
            see(g, x, w);
            bool any = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = take(x[e], id + e, weight.exponent(x[e]));
                any |= in, w[e] = in ? w[e] : 0.f;
            }
            WeightSum of;
            of.add(w);
            const u64 sum = __any_sync(~0u, any) ? of.warp_sum() : 0;
            if (lane == 0) sums[g] = sum;
        });
    };
    // the sums of the units' weights
    auto sum_units = [&](auto take) {
        if constexpr (STREAM) {
            sum_groups_and(groups_ahead, [](int, const float (&)[4], const float (&)[4]) {}, take);
        } else {
            WeightSum mine;
            weigh_stretch([&](const float (&x)[4], float (&w)[4], int id) {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = take(x[e], id + e, weight.exponent(x[e])) ? w[e] : 0.f;
                mine.add(w);
            });
            sums[tid] = mine.sum();
        }
    };
    auto clear_units = [&] {
        for (int g = tid; g < units; g += NT) sums[g] = 0;
        __syncthreads();
    };
    // the CTA's sum, for every thread
    auto block_sum = [&](u64 v) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
        __syncthreads();
        if (lane == 0) sm.part[warp] = v;
        __syncthreads();
        v = sm.part[lane % W];
#pragma unroll
        for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
        return v;
    };
    // inclusive running sum over the CTA's threads
    auto block_scan = [&](u64 v) {
        v = warp_scan(v);
        __syncthreads();
        if (lane == 31) sm.part[warp] = v;
        __syncthreads();
        u64 before = lane < warp ? sm.part[lane] : 0;
#pragma unroll
        for (int o = 16; o; o >>= 1) before += __shfl_xor_sync(~0u, before, o);
        return v + before;
    };
    // a sum over the cluster's threads, for all of them
    auto whole_sum = [&](u64 v) {
        const u64 *const all = tell(block_sum(v));
        v = 0;
        for (int c = 0; c < C; ++c) v += all[c];
        return v;
    };
    // sum of what is told of the kept tokens up to `last` in the order, in the whole row
    auto upto = [&](u64 last, auto of) {
        u64 s = 0;
        groups([&](int, const float (&x)[4], int id) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (kept(x[e], id + e) && order_of(key_of(x[e]), id + e) <= last) s += of(x[e]);
        });
        return whole_sum(s);
    };
    auto one_of = [](float) { return (u64)1; };
    auto weight_of = [&](float x) { return weight(x); };
    // The last token of the shortest start of the kept ones that reaches `want` (mass or number), by bisection: for rows with
    // more candidates than the list takes, of equal or nearly equal values at the cut.
    auto bisect = [&](u64 want, auto of) {
        u64 lo = order_of(key_of(top), 0), hi = order_of(key_of(cut), min(cut_id, (1 << kIdBits) - 1));   // sum(lo - 1) < want <= sum(hi)
        while (lo < hi) {
            const u64 m = lo + (hi - lo) / 2;
            if (upto(m, of) >= want) hi = m;
            else lo = m + 1;
        }
        return lo;
    };
    // The histogram's bin, by bins from 0 down in value, that `want` falls into: before (the sum ahead of it) and its own
    // sum, for every thread; -1 where the sum of all is less. What every CTA of the cluster counted is added.
    auto find_bin = [&](auto masses, auto want_of, u64 &want, u64 &before, u64 &own_sum) {
        sync();
        constexpr int Q = BINS / NT;
        u64 v[Q] = {};
#pragma unroll
        for (int c = 0; c < (ONE ? 1 : 8); ++c)
            if (c < C) {
                const Sh &o = peer(c);
#pragma unroll
                for (int k = 0; k < (masses ? F::REP : 1); ++k)
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const int b = tid * Q + q;
                        v[q] += o.h[k][0][b];
                        if constexpr (masses) v[q] += ((u64)o.h[k][1][b] << 15) + ((u64)o.h[k][2][b] << 30);
                    }
            }
        u64 mine = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) mine += v[q];
        const u64 run = block_scan(mine);
        if (tid == 0) sm.at = -1;
        if (tid == NT - 1) sm.total = run;
        __syncthreads();
        want = want_of(sm.total);
        u64 at = run - mine;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if (at < want && want <= at + v[q]) sm.at = tid * Q + q, sm.above = at, sm.part[0] = v[q];
            at += v[q];
        }
        __syncthreads();
        before = sm.above, own_sum = sm.part[0];
        return sm.at;
    };
    auto reset = [&] {   // histogram and list empty again
        sync();
        empty();
        if (tid == 0) sm.n_list = 0;
        __syncthreads();
    };
    // Candidates of a group, those that take(value) says, into the CTA's list, a place for the whole warp at once; then all of
    // them into that of the cluster's first CTA, if they fit: their number.
    auto push4 = [&](const float (&x)[4], int id, auto take) {
        unsigned is[4];
        int n = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            is[e] = __ballot_sync(~0u, take(e));
            n += __popc(is[e]);
        }
        if (n == 0) return;
        int at = 0;
        if (lane == 0) at = atomicAdd(&sm.n_list, n);
        at = __shfl_sync(~0u, at, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = at + __popc(is[e] & ((1u << lane) - 1));
            if ((is[e] >> lane & 1) && i < LIST) sm.list[i] = order_of(key_of(x[e]), id + e);
            at += __popc(is[e]);
        }
    };
    auto push = [&](float x, int id) {   // (one)
        const int i = atomicAdd(&sm.n_list, 1);
        if (i < LIST) sm.list[i] = order_of(key_of(x), id);
    };
    auto pushed = [&] {
        sync();
        if (ONE || C == 1) return sm.n_list;
        int all = 0, at = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c < C) {
                const int n = peer(c).n_list;
                all += n;
                if (c < rank) at += n;
            }
        if (rank && all <= LIST)
            for (int i = tid; i < sm.n_list; i += NT) peer(0).list[at + i] = sm.list[i];
        sync();
        return all;
    };
    // A long row's threads note the candidates each their own by place, and then put them in one line.
    constexpr int MOST = sizeof(sm.h) / NT;   // a thread's
    const bool by_notes = STREAM && NG <= 64 * W;
    uint8_t *const notes = reinterpret_cast<uint8_t *>(sm.h) + tid;   // (no histogram is in use meanwhile)
    int n_notes = 0;
    auto note = [&](int g, int e) {
        if (n_notes < MOST) notes[n_notes * NT] = (uint8_t)(g / W * 4 + e);
        ++n_notes;
    };
    auto noted = [&] {
        const bool over = __syncthreads_or(n_notes > MOST);
        const int end = (int)block_scan(n_notes), at = end - n_notes;
        if (tid == NT - 1) sm.n_list = end;
        __syncthreads();
        const int all = sm.n_list;
        if (over || all > LIST) return LIST + 1;
#pragma unroll 4
        for (int k = 0; k < n_notes; ++k) {
            const int one = notes[k * NT], id = (warp + (one >> 2) * W) * kGroup + lane * 4 + (one & 3) - lead;
            sm.list[at + k] = order_of(key_of((float)row[id]), id);
        }
        __syncthreads();
        return all;
    };
    // All tokens from a value on into the list, by way of every four or the high groups' (each): their number, above LIST where
    // they do not fit. others(x) sees what is visited.
    auto gather = [&](float from, auto each, auto others) {
        if constexpr (STREAM)
            if (by_notes) {
                each([&](int g, const float (&x)[4], int) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (x[e] >= from) note(g, e);
                    others(x);
                });
                return noted();
            }
        each([&](int, const float (&x)[4], int id) {
            if (__any_sync(~0u, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) >= from)) push4(x, id, [&](int e) { return x[e] >= from; });
            others(x);
        });
        return pushed();
    };
    auto sort = [&](u64 *list, int n) {   // room for a power of two
        int n2 = 16;
        while (n2 < n) n2 *= 2;
        if (n2 <= NT / 2) {   // short: an entry's place is how many are before it, counted by several threads
            const int lanes = min(NT / n2, 32), i = tid / lanes, k0 = tid % lanes;
            const u64 e = i < n ? list[i] : ~0ull;
            int at = 0;
            for (int k = k0; k < n; k += lanes) at += list[k] < e;
            for (int o = lanes / 2; o; o >>= 1) at += __shfl_xor_sync(~0u, at, o);
            __syncthreads();
            if (i < n && k0 == 0) list[at] = e;
            __syncthreads();
            return;
        }
        for (int i = tid + n; i < n2; i += NT) list[i] = ~0ull;
        __syncthreads();
        for (int size = 2; size <= n2; size *= 2)
            for (int half = size / 2; half; half /= 2) {
                for (int k = tid; k < n2 / 2; k += NT) {
                    const int i = 2 * k - (k & (half - 1)), j = i + half;
                    const u64 x = list[i], y = list[j];
                    if ((x > y) == ((i & size) == 0)) list[i] = y, list[j] = x;
                }
                // (32 pairs half 32 or less apart are a warp's own 64 entries)
                if (half > 32 || (half == 1 && size >= 64)) __syncthreads();
                else __syncwarp();
            }
        __syncthreads();
    };
    auto id_of = [&](u64 order) { return (int)(order & ((1 << kIdBits) - 1)); };
    auto value_at = [&](u64 order) { return value_of(~(uint32_t)(order >> kIdBits)); };
    const bool by_p = top_p < 1.f && !greedy, by_k = top_k > 0 && top_k < V && !greedy;
    // How far a difference between a sum of weights and f times all of them, near 0, may be off: S the latter. (Of a part A and
    // the rest B, A - f (A + B) = (1 - f) A - f B, and both are f (1 - f) S there; and what is cut off below the units.)
    auto slack = [&](u64 S, float f) { return (u64)(__ull2float_rn(S) * (2.f * kOff * f * (1.f - f))) + V; };
    u64 mass = 0;             // of all that top-p takes its part of
    bool cut_unsure = false;  // whether its cut is one by less than that
    auto threshold = [&](u64 S) {   // ceil(top_p S): a token is kept by top-p where the mass before it is below this
        mass = S;
        const u64 p = part64(fminf(fmaxf(top_p, 0.f), 0.99999994f));
        return max(1ull, __umul64hi(p, S) + (p * S != 0));
    };
    // whether a cut is: w the last kept token's weight, upto the sum with it, both in units that P and so the threshold is in
    // (ahead: what they leave out)
    auto near_cut = [&](u64 w, u64 upto, u64 P, u64 ahead) {
        const u64 E = slack(mass, fminf(fmaxf(top_p, 0.f), 1.f));
        return (ahead + upto > w && upto - w + E >= P) || upto < P + E;
    };
    // Of a sorted list's first n entries, whose sum comes after `ahead` (and after `above`, which P leaves out): how many are kept
    // where a token is that has less than P(their sum) before it; their sum, and whether that is near.
    auto kept_of = [&](const u64 *list, int n, u64 ahead, u64 above, auto P_of, u64 &sum) {
        if (n <= NT) {
            const u64 w = tid < n ? weight(value_at(list[tid])) : 0, run = block_scan(w);
            if (tid == NT - 1) sm.total = run;
            __syncthreads();
            const u64 P = P_of(sm.total);
            const int m = __syncthreads_count(tid < n && ahead + run - w < P);
            if (tid == m - 1) sm.kept = run, sm.cut_unsure = by_p && near_cut(w, ahead + run, P, above);
            __syncthreads();
            sum = sm.kept;
            return m;
        }
        const int q = (n + NT - 1) / NT, i0 = min(n, tid * q), i1 = min(n, i0 + q);   // a thread's entries
        u64 mine = 0;
        for (int i = i0; i < i1; ++i) mine += weight(value_at(list[i]));
        const u64 run = block_scan(mine);
        if (tid == NT - 1) sm.total = run;
        if (tid == 0) sm.n_kept = 0;
        __syncthreads();
        const u64 P = P_of(sm.total);
        u64 at = ahead + run - mine;
        for (int i = i0; i < i1; ++i) {
            if (at >= P) break;
            const u64 w = weight(value_at(list[i]));
            at += w;
            if (i == n - 1 || at >= P) sm.n_kept = i + 1, sm.kept = at - ahead, sm.cut_unsure = by_p && near_cut(w, at, P, above);
        }
        __syncthreads();
        sum = sm.kept;
        return sm.n_kept;
    };
    // the segment's share of a list's entries up to `last` added to the groups' sums
    auto add_listed = [&](const u64 *list, int n, u64 last) {
        for (int i = tid; i < n; i += NT) {
            const u64 e = list[i];
            const int pos = id_of(e) + lead - base;
            if (e <= last && pos >= 0 && pos < SL) add64(&sums[pos / unit], weight(value_at(e)));
        }
    };

    // Of the list's n entries up to `most` in the order, all from one value down to another (`ahead` of them the tokens of more
    // than that): the last one of the shortest start that reaches want_of(their number or mass); 0 where none does. A histogram
    // and its bin's entries, so that a long list is not sorted.
    auto choose = [&](int n, u64 most, float to, float from, u64 ahead, auto masses, auto want_of) {
        reset();   // (the list stays)
        const float y0 = weight.exponent(to), scale = (BINS - 1) / (weight.exponent(from) - y0 - 0.01f);
        // (held in float to the last bin, whatever the distance: the sum with 1.5 * 2^23 is a whole number in its lower bits)
        auto bin = [&](float x) {
            return __float_as_int(fminf((weight.exponent(x) - y0) * scale, (float)(BINS - 1)) + 12582912.f) & (2 * BINS - 1);
        };
        uint32_t(*const h)[BINS] = sm.h[masses ? warp % F::REP : 0];
        for (int i = tid; i < n; i += NT) {
            const u64 e = sm.list[i];
            if (e > most) continue;
            const float x = value_at(e);
            const int at = bin(x);
            if constexpr (masses) {
                const u64 w = weight(x);
                atomicAdd(&h[0][at], (uint32_t)w & 0x7fffu);
                atomicAdd(&h[1][at], (uint32_t)(w >> 15) & 0x7fffu);
                if (w >> 30) atomicAdd(&h[2][at], (uint32_t)(w >> 30));
            } else {
                atomicAdd(&h[0][at], 1u);
            }
        }
        u64 want, before, own_sum, sum;
        const int at = find_bin(masses, want_of, want, before, own_sum);
        if (at < 0) return 0ull;
        u64 *const some_of = reinterpret_cast<u64 *>(sm.h);   // the bin's entries
        constexpr int ROOM = 2048;
        static_assert(ROOM * 8 <= sizeof(sm.h) || !STREAM);
        for (int i = tid; i < n; i += NT) {
            const u64 e = sm.list[i];
            if (e <= most && bin(value_at(e)) == at) {
                const int k = atomicAdd(&sm.n_list, 1);
                if (k < ROOM) some_of[k] = e;
            }
        }
        __syncthreads();
        const int m = sm.n_list;
        if (m > ROOM) {
            cut_at(min(most, order_of(key_of(from), (1 << kIdBits) - 1)));
            if constexpr (masses) cut_unsure = true;   // (how near it is is not known)
            if constexpr (masses) return bisect(ahead + want, weight_of);
            else return bisect(ahead + want, one_of);
        }
        sort(some_of, m);
        if constexpr (masses) {
            const u64 last = some_of[kept_of(some_of, m, before, ahead, [&](u64) { return want; }, sum) - 1];
            cut_unsure = sm.cut_unsure;
            return last;
        } else return some_of[(int)(want - before) - 1];
    };

    // What exact sums are asked for, where all weights sum to S: their exact ones, up to 1.42 times as much, fit 64 bits.
    auto drop_of = [&](u64 S) { return max(0, 64 - __clzll(S) - kUnitBits - 1); };
    // The cut of top-p among the tokens that are kept so far, by exact weights, from one that is off by a few tokens at most: their
    // sum and that of those before the cut once, and then from token to token; where these are many, by bisection.
    auto exact_cut = [&](u64 last) {
        const int drop = drop_of(mass);
        auto of = [&](float x) { return weight.exact(x, drop); };
        u64 S = 0, before = 0;
        groups([&](int, const float (&x)[4], int id) {
            float all[4], some[4];
            bool any = false, each = true;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                all[e] = kept(x[e], id + e) ? x[e] : -INFINITY;
                const bool is = order_of(key_of(x[e]), id + e) < last;
                some[e] = is ? all[e] : -INFINITY;
                any |= some[e] > -INFINITY, each &= some[e] == all[e];
            }
            const u64 w = weight.exact(all[0], all[1], all[2], all[3], drop);
            S += w;
            if (each) before += w;
            else if (any) before += weight.exact(some[0], some[1], some[2], some[3], drop);
        });
        S = whole_sum(S), before = whole_sum(before);
        const u64 P = threshold(S);
        // the kept token next to `at` in the order, before or after it (~0: there is none)
        auto next_to = [&](u64 at, bool after) {
            u64 best = after ? ~0ull : 0;
            groups([&](int, const float (&x)[4], int id) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const u64 o = order_of(key_of(x[e]), id + e);
                    if (kept(x[e], id + e) && (after ? o > at && o < best : o < at && o >= best)) best = o;
                }
            });
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const u64 y = __shfl_xor_sync(~0u, best, o);
                best = after ? min(best, y) : max(best, y);
            }
            __syncthreads();
            if (lane == 0) sm.part[warp] = best;
            __syncthreads();
            for (int w = 0; w < W; ++w) best = after ? min(best, sm.part[w]) : max(best, sm.part[w]);
            const u64 *const all = tell(best);
            for (int c = 0; c < C; ++c) best = after ? min(best, all[c]) : max(best, all[c]);
            return best;
        };
        constexpr int MANY = 32;
        int steps = 0;
        while (before >= P && ++steps <= MANY) {
            last = next_to(last, false);
            before -= of(value_at(last));
        }
        while (before < P && ++steps <= MANY) {
            const u64 with = before + of(value_at(last));
            if (with >= P) return last;
            const u64 next = next_to(last, true);
            if (next == ~0ull) return last;
            before = with, last = next;
        }
        return bisect(P, of);
    };

    u64 S = 0;                // the sum of all kept weights
    bool listed = false;      // all kept tokens are in the list,
    int n_list = 0;           // of this length: those up to
    u64 last = ~0ull;         // this place in the order
    bool summed = false;      // sums are those of the kept tokens
    bool drawn = false;
    // ~0: all that are kept so far
    auto cut_again = [&](u64 most) {
        if (most != ~0ull) cut_at(most);
        else cut = low, cut_id = 1 << kIdBits;
    };
    // Values in equal bins from the top down: how far down the threads' largest of a number `want` lie. At least as many
    // tokens do, and few more.
    const float span = top - fmaxf(low, top - 64.f * fmaxf(temp, 0.25f)), vscale = span > 0.f ? (BINS - 1) / span : 0.f;
    auto vbin = [&](float x) { return (int)fminf((top - x) * vscale, (float)(BINS - 1)); };
    auto sample_bin = [&](u64 number) {
        if (number <= NT * C / 2) {   // one a thread is enough
            own[0] = fmaxf(fmaxf(own[0], own[1]), fmaxf(own[2], own[3]));
            own[1] = own[2] = own[3] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (own[e] >= low) atomicAdd(&sm.h[0][0][vbin(own[e])], 1u);
        u64 want, before, own_sum;
        const int b = find_bin(std::false_type(), [&](u64) { return number; }, want, before, own_sum);
        return b < BINS - 1 ? b : -1;
    };
    // Values between which the last token kept by top-p alone lies, most likely: from the largest of each quarter of a thread's
    // elements, which tell the number of tokens above a value where that is small (of n, none is with (1 - f)^n), and from a
    // sample of all where it is not. Right is what is then counted; an estimate that is off costs time. Counts of the tokens
    // from lo on and from hi on.
    struct Range {
        float lo, hi;
        int n_lo, n_hi;
    };
    auto estimate = [&] {
        Range z{low, top, 1 << 30, 0};
        if constexpr (STREAM) {
            constexpr float FIX = 65536.f, EIGHTHS = 8.f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (own[e] >= low) atomicAdd(&sm.h[0][0][vbin(own[e])], 1u);
            const int chunks = (v_hi + 31) / 32;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int v = (4 * warp + 2 * k + 1) * chunks / (4 * W) * 32 + lane;
                if (v < v_lo || v >= v_hi) continue;
                const uint4 x = pieces[v];
#pragma unroll
                for (int i = 0; i < VE; i += 4) {
                    float f[4];
                    load4(reinterpret_cast<const T *>(&x) + i, f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) atomicAdd(&sm.h[0][1][vbin(f[e])], 1u);
                }
            }
            __syncthreads();
            const u64 both = sm.h[0][0][tid] | (u64)sm.h[0][1][tid] << 32, run = block_scan(both);   // (a bin a thread)
            if (tid == NT - 1) sm.total = run;
            if (tid == 0) sm.at = -1, sm.n_kept = 0;
            __syncthreads();
            const float samples = fmaxf(1.f, (float)(uint32_t)(sm.total >> 32));
            auto share = [&](u64 r) { return 1.f - ex2(__log2f(fmaxf(1.f - (float)(uint32_t)r / (4 * NT), 1e-6f)) * (4.f * NT) / V); };
            const float f = (uint32_t)run < 3 * NT ? share(run) - share(run - both) : (float)(uint32_t)(both >> 32) / samples;
            const float n = f * V, mass = n * ex2(-(tid + 0.5f) / vscale * by * ch);
            // mass and number in one sum
            const u64 mine = (u64)(mass * FIX) << 24 | (u64)(n * EIGHTHS), upto = block_scan(mine), ahead = upto - mine;
            if (tid == NT - 1) sm.total = upto;
            __syncthreads();
            const float S = (float)(sm.total >> 24), p = fminf(fmaxf(top_p, 0.f), 1.f), off = fminf(0.02f, 0.15f * fminf(p, 1.f - p));
            const float m0 = (float)(ahead >> 24), m1 = (float)(upto >> 24);
            if (m0 < (p + off) * S && (p + off) * S <= m1) sm.at = tid, sm.above = upto & 0xffffff;
            if (m0 < (p - off) * S && (p - off) * S <= m1) sm.n_kept = tid, sm.kept = ahead & 0xffffff;
            __syncthreads();
            if (sm.at >= 0) {
                z.lo = top - (sm.at + 1) / vscale, z.n_lo = (int)sm.above / 8;
                z.hi = top - sm.n_kept / vscale, z.n_hi = sm.n_kept ? (int)sm.kept / 8 : 0;
            }
            __syncthreads();
        }
        return z;
    };
    bool cut_found = false;
    if (greedy) {
        u64 first = ~0ull;
        high_groups(top, [&](int, const float (&x)[4], int id) {
#pragma unroll
            for (int e = 3; e >= 0; --e)
                if (x[e] == top) first = min(first, order_of(key_of(top), id + e));
        });
#pragma unroll
        for (int o = 16; o; o >>= 1) first = min(first, __shfl_xor_sync(~0u, first, o));
        if (lane == 0) sm.part[warp] = first;
        __syncthreads();
        for (int w = 0; w < W; ++w) first = min(first, sm.part[w]);
        const u64 *const all = tell(first);
        for (int c = 0; c < C; ++c) first = min(first, all[c]);
        cut_at(first);
        S = 1ull << kUnitBits;
        drawn = true;
        if (a.token && rank == 0 && tid == 0) a.token[r] = cut_id;
    } else if (by_k || min_p > 0.f) {
        // ---- top-k and min-p
        u64 want, before = 0, own_sum = 0;
        float list_from = low;
        int b = -1;
        if (by_k && top_k < SORT && top_k <= 2 * NT * C) b = sample_bin(top_k);
        if (b >= 0 || min_p > 0.f) {
            // no lower than any value of the bins up to b
            const float from = b < 0 || vscale == 0.f ? low : fmaxf(low, top - (b + 1) / vscale * 1.00001f - fabsf(top) * 1e-6f);
            n_list = gather(from, [&](auto f) { high_groups(from, f); }, [](const float (&)[4]) {});
            listed = n_list <= LIST;
            list_from = from;
        }
        if (by_k && !listed) {   // bins of every token: all candidates in the k-th one's, with the bins above it where they fit
            reset();
            groups([&](int, const float (&x)[4], int) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (x[e] >= low) atomicAdd(&sm.h[0][0][vbin(x[e])], 1u);
            });
            b = find_bin(std::false_type(), [&](u64) { return (u64)top_k; }, want, before, own_sum);
            listed = b >= 0 && before + own_sum <= SORT;
            // (the last bin has whatever is below it)
            if (listed)
                list_from = vscale == 0.f || b == BINS - 1 ? low : fmaxf(low, top - (b + 1) / vscale * 1.00001f - fabsf(top) * 1e-6f);
            if (b >= 0 && own_sum > SORT) cut_at(bisect(top_k, one_of));
            else if (b >= 0) {   // (otherwise fewer than k tokens: all are kept)
                groups([&](int, const float (&x)[4], int id) {
                    push4(x, id, [&](int e) { return x[e] >= low && (listed ? vbin(x[e]) <= b : vbin(x[e]) == b); });
                });
                n_list = pushed();
                if (!listed) {
                    if (rank == 0) {
                        sort(sm.list, n_list);
                        if (tid < C) peer(tid).cut = sm.list[top_k - (int)before - 1];
                    }
                    sync();
                    cut_at(sm.cut);
                }
            }
        }
        if (STREAM && listed && n_list > NT) {
            // ---- a long list's
            last = ~0ull;
            // (fewer than top_k where min-p keeps fewer: then all of them, and the cut stays at its bound)
            if (by_k && n_list >= top_k) last = choose(n_list, last, top, list_from, 0, std::false_type(), [&](u64) { return (u64)top_k; });
            const u64 most = last;
            if (by_p) last = choose(n_list, last, top, list_from, 0, std::true_type(), threshold);
            if (cut_unsure) {
                cut_again(most);
            } else {
                if (last != ~0ull) cut_at(last);
                __syncthreads();
                clear_units();
                add_listed(sm.list, n_list, last);
                summed = true;
            }
        } else if (listed) {
            // ---- the list's kept entries, in the cluster's first CTA; and the token, if they are few, by every entry's thread
            if (rank == 0) {
                int n = n_list;
                if (by_k || by_p) sort(sm.list, n);
                if (by_k) n = min(n, top_k);
                const u64 most = n < n_list ? sm.list[n - 1] : ~0ull;
                u64 sum;
                n = kept_of(sm.list, n, 0, 0, [&](u64 all) { return by_p ? threshold(all) : (mass = all, ~0ull); }, sum);
                if (n <= NT / 4) {
                    u64 *const w_s = reinterpret_cast<u64 *>(sm.h);
                    const u64 e = tid < n ? sm.list[tid] : 0, w = tid < n ? weight(value_at(e)) : 0;
                    if (tid < n) w_s[tid] = w;
                    __syncthreads();
                    if (a.token && tid < n) {
                        const u64 place = __umul64hi(part64(u), sum);
                        u64 at = 0;
#pragma unroll 4
                        for (int i = 0; i < n; ++i) at += id_of(sm.list[i]) < id_of(e) ? w_s[i] : 0;
                        if (at <= place && place < at + w) {
                            const u64 E = slack(sum, u);
                            a.token[r] = id_of(e);
                            if (place - at < E || at + w - place <= E)
                                for (int c = 0; c < C; ++c) peer(c).draw_unsure = true;
                        }
                    }
                }
                if (tid < C) {
                    Sh &o = peer(tid);
                    o.n_kept = n, o.kept = sum, o.cut = by_k || by_p ? sm.list[n - 1] : ~0ull;
                    o.most = most, o.total = mass, o.cut_unsure = sm.cut_unsure;
                }
            }
            sync();
            S = sm.kept, last = sm.cut, mass = sm.total;
            cut_unsure = sm.cut_unsure;
            if (cut_unsure) {
                cut_again(sm.most);
            } else {
                if (by_k || by_p) cut_at(last);
                if (sm.n_kept <= NT / 4 && !sm.draw_unsure) drawn = true;
                else {
                    clear_units();
                    add_listed(peer(0).list, n_list, last);
                    summed = true;
                }
            }
        }
    }
    if constexpr (STREAM)
        if (bound && by_p) {
            // ---- top-p alone, where the cut lies between two values: the list has the tokens between them, or all from the lower
            // one on where these fit too; what is above and below is only summed
            constexpr int FITS = LIST * 4 / 5;
            Range z = vscale > 0.f ? estimate() : Range{low, top, 1 << 30, 0};
            z.lo = fmaxf(low, z.lo);   // (only tokens are in)
            WeightSum below;
            u64 rest = 0;
            auto rest_of = [&](const float (&x)[4], const float (&w)[4]) {
                float of[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) of[e] = x[e] >= z.lo ? 0.f : w[e];
                below.add(of);
            };
            if (z.n_lo <= FITS) {
                n_list = gather(z.lo, groups_ahead, [&](const float (&x)[4]) {
                    float w[4];
                    weight.four(x, w);
                    rest_of(x, w);
                });
                rest = block_sum(below.sum());
                if (n_list <= LIST) {
                    last = choose(n_list, ~0ull, top, z.lo, 0, std::true_type(), [&](u64 mass) { return threshold(mass + rest); });
                    listed = cut_found = last != 0;
                }
                if (listed) clear_units();
            } else if (z.n_lo - z.n_hi <= FITS) {
                sum_groups_and(groups, [&](int g, const float (&x)[4], const float (&w)[4]) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (x[e] >= z.lo && x[e] <= z.hi) {
                            if (by_notes) note(g, e);
                            else push(x[e], g * kGroup + lane * 4 + e - lead);
                        }
                    rest_of(x, w);
                }, [&](float v, int, float) { return v > z.hi; });
                rest = block_sum(below.sum());
                u64 above = 0;
                for (int g = tid; g < NG; g += NT) above += sums[g];
                above = block_sum(above);
                n_list = by_notes ? noted() : sm.n_list;
                if (n_list <= LIST) {
                    last = choose(n_list, ~0ull, z.hi, z.lo, above, std::true_type(), [&](u64 mass) {
                        const u64 P = threshold(above + mass + rest);
                        return P > above ? P - above : ~0ull;
                    });
                    cut_found = last != 0;
                }
            }
            if (cut_unsure) {
                cut_again(~0ull);
            } else if (cut_found) {
                cut_at(last);
                add_listed(sm.list, n_list, last);
                summed = true;
            } else {
                reset();
            }
        }
    if (by_p && !listed && !cut_found && !cut_unsure) {
        if (by_k || min_p > 0.f) reset();
        // ---- top-p: exact sums of weights in equal bins of the exponent; tokens so light that all of them together make
        // less than 1 - top_p of the whole are only added up
        const float least =
            fminf(-0.01f, fmaxf(-41.f, log2f(fmaxf(1.f - top_p, 1e-9f)) + (bound ? log2f(some) : 0.f) - log2f((float)V) - 0.02f));
        const float scale = (BINS - 1) / least;
        // bin BINS - 1: from least down. (The sum with 1.5 * 2^23 is a whole number in its lower bits.)
        auto bin = [&](float y) {
            return y <= least ? BINS - 1 : min(BINS - 2, __float_as_int(fmaf(y, scale, 12582912.f)) & (2 * BINS - 1));
        };
        u64 rest = 0;
        uint32_t(*const h)[BINS] = sm.h[warp % F::REP];
        auto count = [&](float y, u64 w) {
            const int b = bin(y);
            if (b == BINS - 1) rest += w;
            else {
                atomicAdd(&h[0][b], (uint32_t)w & 0x7fffu);
                atomicAdd(&h[1][b], (uint32_t)(w >> 15) & 0x7fffu);
                if (w >> 30) atomicAdd(&h[2][b], (uint32_t)(w >> 30));
            }
        };
        auto spread = [&](auto take) {
            auto count4 = [&](const float (&x)[4], const float (&w)[4], int id) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (take(x[e], id + e, 0.f)) count(weight.exponent(x[e]), Weights::whole(w[e]));
            };
            if constexpr (STREAM) {
                groups([&](int, const float (&x)[4], int id) {
                    float w[4];
                    weight.four(x, w);
                    count4(x, w, id);
                });
            } else {
                weigh_stretch(count4);
            }
        };
        if (bound) spread(all_of_them);
        else spread(kept_of_them);
        rest = block_sum(rest);
        if (tid < 3) sm.h[0][tid][BINS - 1] = tid == 0 ? (uint32_t)rest & 0x7fffu : tid == 1 ? (uint32_t)(rest >> 15) & 0x7fffu : (uint32_t)(rest >> 30);
        u64 P, before, own_sum;
        const int b = find_bin(std::true_type(), threshold, P, before, own_sum);
        // sums of what is kept in the bins before, candidates of the bin itself
        sum_units([&](float v, int i, float y) {
            const int at = kept(v, i) ? bin(y) : BINS;
            if (at == b) push(v, i);
            return at < b;
        });
        n_list = pushed();
        if (n_list > SORT) {
            last = bisect(P, weight_of), cut_unsure = true;   // (how near it is is not known)
        } else {
            if (rank == 0) {
                u64 sum;
                sort(sm.list, n_list);
                const int m = kept_of(sm.list, n_list, before, 0, [&](u64) { return P; }, sum);
                if (tid < C) peer(tid).cut = sm.list[m - 1], peer(tid).cut_unsure = sm.cut_unsure;
            }
            sync();
            last = sm.cut, cut_unsure = sm.cut_unsure;
            if (!cut_unsure) {
                cut_at(last);
                add_listed(peer(0).list, n_list, last);
                summed = true;
            }
        }
    }
    if (cut_unsure) {
        cut_at(exact_cut(last));
        listed = false;
    }
    // The group and the token that u falls on, from the sums of the units and the weights that they are of; the sum of all.
    auto draw = [&](auto of, auto E_of) {
        __syncthreads();
        const int share = (units + NT - 1) / NT, g0 = min(units, tid * share), g1 = min(units, g0 + share);   // a thread's units
        u64 mine = 0;
        for (int g = g0; g < g1; ++g) mine += sums[g];
        const u64 run = block_scan(mine);
        if (tid == NT - 1) sm.total = run;
        __syncthreads();
        const u64 *const all = tell(sm.total);
        u64 first = 0, S = 0;
        for (int c = 0; c < C; ++c) {
            if (c < rank) first += all[c];
            S += all[c];
        }
        if (!a.token) return S;
        // the first id at which the running sum is above u S
        const u64 want = __umul64hi(part64(u), S);
        if (first + run - mine <= want && want < first + run) {
            u64 at = first + run - mine;
            int g = g0;
            while (want >= at + sums[g]) at += sums[g++];
            sm.at = g, sm.above = at;
        }
        const bool here = first <= want && want < first + all[rank];
        __syncthreads();
        if (here && warp == 0) {
            const int from = sm.at * unit + lane * 4, id = base + from - lead;
            float x[4];
            u64 w[4], sum = 0;
            if constexpr (STREAM) get4(from, x);
            else four_at(from, min(SL, (sm.at + 1) * unit), x);
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += w[e] = kept(x[e], id + e) ? of(x[e]) : 0;
            u64 at = sm.above + warp_scan(sum) - sum;
            if (at <= want && want < at + sum) {
                const u64 E = E_of(S);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (at <= want && want < at + w[e]) {
                        a.token[r] = id + e;
                        if (want - at < E || at + w[e] - want <= E)
                            for (int c = 0; c < C; ++c) peer(c).draw_unsure = true;
                    }
                    at += w[e];
                }
            }
        }
        return S;
    };
    // The same by exact weights, where the first ones leave it open.
    auto draw_exactly = [&] {
        const int drop = drop_of(S);
        auto of = [&](float x) { return weight.exact(x, drop); };
        auto four_of = [&](const float (&x)[4], int id) {
            float y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = kept(x[e], id + e) ? x[e] : -INFINITY;
            return weight.exact(y[0], y[1], y[2], y[3], drop);
        };
        if constexpr (STREAM) {
            groups([&](int g, const float (&x)[4], int id) {
                const u64 sum = warp_sum(four_of(x, id));
                if (lane == 0) sums[g] = sum;
            });
        } else {
            u64 mine = 0;
            const int i0 = min(SL, tid * unit), i1 = min(SL, i0 + unit);
#pragma unroll 1
            for (int i = i0; i < i1; i += 4) {
                float x[4];
                four_at(i, i1, x);
                mine += four_of(x, base + i - lead);
            }
            sums[tid] = mine;
        }
        draw(of, [](u64) { return (u64)0; });
    };
    if (!drawn) {
        // ---- kept weights, group by group
        if (!summed) {
            if (cut_id == 1 << kIdBits && low == -3.402823466e38f) sum_units(all_of_them);
            else sum_units(kept_of_them);
        }
        S = draw(weight_of, [&](u64 S) { return slack(S, u); });
        if (ONE || C == 1) {   // (a cluster does it at the end, at its last barrier: its rows are in shared memory)
            __syncthreads();
            if (sm.draw_unsure) draw_exactly();
        }
    }
    const float inv = (greedy ? kUnits : __ull2float_rn(weight(top))) / __ull2float_rn(S);
    if (p_to || k_to) {
        if (listed || greedy) {   // few tokens
            __syncthreads();      // (the row may be where they go, and is read no more)
            fill_rows(0.f, TS_DROPPED_LOGIT);
            __syncthreads();
            const Sh &o = peer(0);
            for (int i = tid; i < (greedy ? 1 : n_list); i += NT) {
                if (!greedy && o.list[i] > last) continue;
                const int id = greedy ? cut_id : id_of(o.list[i]), pos = id + lead - base;
                if (pos < 0 || pos >= SL) continue;
                const float x = greedy ? top : value_at(o.list[i]);
                if (p_to) p_to[id] = greedy ? 1.f : weight.real(x, inv);
                if (k_to) k_to[id] = x;
            }
        } else {
            if (STREAM) __syncthreads();   // (the same: the token's group may still be read)
#pragma unroll 4
            for (int v = tid; v < SL / 4; v += NT) {
                float x[4], y[4];
                bool in[4];
                get4(4 * v, x);
                const int p = base + 4 * v - lead;
#pragma unroll
                for (int e = 0; e < 4; ++e) in[e] = kept(x[e], p + e), y[e] = 0.f;
                if (p_to) {
                    if (in[0] | in[1] | in[2] | in[3]) {
                        weight.real4(x, inv, y);
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = in[e] ? y[e] : 0.f;
                    }
                    put4(p_to, p, y);
                }
                if (k_to) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = in[e] ? x[e] : TS_DROPPED_LOGIT;
                    put4(k_to, p, y);
                }
            }
        }
    }
    if (!ONE && C > 1) {
        cluster.sync();   // shared memory that others may still read
        if (!drawn && sm.draw_unsure) {
            draw_exactly();
            cluster.sync();
        }
    }
}

template <Mode M>
size_t smem_of(int SL, int es) {
    const int units = M == kStream ? SL / kGroup : Cfg<M>::NT;
    return kFixed<M> + (size_t)(units + 1) / 2 * 16 + (M == kStream ? 0 : (size_t)SL * es);
}

template <typename T, Mode M>
cudaError_t launch_as(const SampleArgs &a, int C, int SL, cudaStream_t s) {
    constexpr auto kern = k_sample<T, M>;
    const size_t smem = smem_of<M>(SL, sizeof(T));
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.R * C);
    cfg.blockDim = dim3(Cfg<M>::NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    const int pdl = pdl_enabled();
    cfg.attrs = attr + !pdl;
    cfg.numAttrs = pdl + (M == kCluster);
    return cudaLaunchKernelEx(&cfg, kern, a, SL);
}

template <typename T>
cudaError_t launch_rows(const SampleArgs &a, cudaStream_t s) {
    auto seg = [&](int C) { return ((a.V + 16 / (int)sizeof(T) - 1 + C - 1) / C + kGroup - 1) / kGroup * kGroup; };
    // The fewest CTAs a row whose segments let two of them share an SM (228 KB, of which each takes one for itself); more where
    // there are few rows, while every CTA has an SM. (Two CTAs a row and four, 39 to 65 rows of 50272, from the whole distribution
    // 10.2 to 11.0 and 10.8 to 11.6 us, top-k 50 13.0 to 13.8 and 13.6 to 14.5, top-p 0.9 30.5 to 31.1 and 29.1 to 30.0, min-p 13.4
    // to 14.2 and 13.1 to 13.9; 76 rows 16.6 and 19.7, 14.5 and 24.0, 31.9 and 49.1, 15.1 and 21.6; 32000 alike.)
    constexpr size_t kHalf = (228 / 2 - 1) * 1024;
    int C = 1;
    while (C < 8 && smem_of<kCluster>(seg(C), sizeof(T)) > kHalf) C *= 2;
    // Filtered rows, more than there are SMs: a CTA a row, from L2 (cluster and CTA: 160 rows of 50272 with top-k 50 28 and 23
    // us, top-p 0.9 65 and 53, settings by row and distributions 58 and 68; 300 rows 35 and 25, 87 and 63, 89 and 93; 1024 rows
    // 109 and 80, 259 and 163, 190 and 138; 100 rows 17.5 and 18, 42 and 40, 53 and 61). Not filtered, a row is read from shared
    // memory (100 rows 21 and 27 us, 300 rows 42 and 53, 1024 rows 101 and 100).
    if (C > 1 && a.R > num_sms() && (a.top_k || a.top_p || a.min_p)) return launch_as<T, kStream>(a, 1, seg(1), s);
    while (C < 8 && 2LL * a.R * C <= num_sms() && seg(2 * C) >= 2048) C *= 2;
    // Short rows, where there are more than the SMs hold at once in large CTAs (small CTAs and large: settings by row and
    // distributions, 1000 tokens, 300 rows 12.3 and 13.0 us, 1200 rows 17 and 46; 4000 tokens, 300 rows 30 and 21.5, 450 rows 31
    // and 30, 1200 rows 41 and 60).
    if (C == 1 && a.V <= 4096 && (a.V <= 512 || a.R >= num_sms() + a.V / 8)) return launch_as<T, kSmall>(a, 1, seg(1), s);
    return launch_as<T, kCluster>(a, C, seg(C), s);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, ts_dtype dt, cudaStream_t s) {
    return dt == TS_BF16 ? launch_rows<__nv_bfloat16>(a, s) : launch_rows<float>(a, s);
}

}  // namespace ts
