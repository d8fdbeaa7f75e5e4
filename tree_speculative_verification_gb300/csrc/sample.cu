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
// wrongly about once in a thousand draws. So weights are whole numbers, the
// largest 2^40 (weight): their sums are exact, whatever the order, up to 2^18
// tokens.
#include <cuda_bf16.h>
#include <math.h>

#include "decode.cuh"

namespace ts {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr uint32_t kKeyLowest = 0x00800000u;   // key of the lowest finite number
typedef unsigned long long u64;

// Whole numbers in the order of the floats (-0 counts as 0).
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// 2^(j / 8) as two floats each.
__constant__ float kRootHi[8] = {0x1.0000000000000p+0f, 0x1.172b840000000p+0f, 0x1.306fe00000000p+0f, 0x1.4bfdae0000000p+0f,
                                 0x1.6a09e60000000p+0f, 0x1.8ace540000000p+0f, 0x1.ae89fa0000000p+0f, 0x1.d5818e0000000p+0f};
__constant__ float kRootLo[8] = {0x0.0p+0f, -0x1.c157420000000p-27f, 0x1.4636e20000000p-25f, -0x1.593abc0000000p-25f,
                                 0x1.9fcef40000000p-26f, 0x1.15506e0000000p-27f, -0x1.a94b140000000p-26f, -0x1.822dbc0000000p-27f};

// exp((x - top) / T) in units of 2^-40, to the unit and some 2^-38 of itself.
// y = (x - top) log2(e) / T as a sum of two floats (the difference and the
// products by their exact errors), y = n + j / 8 + g, and
// 2^y = 2^n 2^(j/8) (1 + t + t^2 / 2 + ...), t = g ln 2, |t| < 0.0434: the first
// two terms as sums of two floats, the rest (below 2^-16) in one.
struct Weights {
    float top, ch, cl;   // log2(e) / T = ch + cl
    __device__ __forceinline__ u64 operator()(float x) const {
        if (x == top) return 1ull << 40;
        const float dh = x - top, bb = dh - x, dl = (x - (dh - bb)) - (top + bb);
        const float yh = dh * ch;
        if (!(yh > -44.f)) return 0;
        const float yl = fmaf(dh, ch, -yh) + fmaf(dh, cl, dl * ch);
        const float n8 = rintf(yh * 8.f), f = fmaf(n8, -0.125f, yh);
        const float gh = f + yl, gl = yl - (gh - f);
        const float L = 0.693147182464599609375f, Ll = -1.904654299957767e-09f;   // ln 2
        const float th = gh * L, tl = fmaf(gh, L, -th) + fmaf(gh, Ll, gl * L);
        const float hh = 0.5f * th, sh = hh * th, sl = fmaf(hh, th, -sh) + th * tl;
        const float r = th * th * th * fmaf(th, fmaf(th, fmaf(th, 1.f / 720, 1.f / 120), 1.f / 24), 1.f / 6);
        const float ph = th + sh, pl = (sh - (ph - th)) + ((tl + sl) + r);
        const int m = (int)n8, j = m & 7, n = m >> 3;                             // m = 8 n + j
        const float Rh = kRootHi[j], Rl = kRootLo[j];
        const float z = Rh * ph, hi = Rh + z, lo = (z - (hi - Rh)) + (fmaf(Rh, ph, -z) + fmaf(Rh, pl, fmaf(Rl, ph, Rl)));
        // hi in [0.95, 2.1): a whole number of 2^-24; in units of 2^-42, then 2^(n - 40)
        const long long v = ((long long)(int)(hi * 16777216.f) << 18) + __float2int_rn(lo * 4398046511104.f);
        const int sft = 2 - n;
        return (u64)((v + (1ll << (sft - 1))) >> sft);
    }
    // The same as a float, to some 2^-22 of itself.
    __device__ __forceinline__ float real(float x) const {
        const float dh = x - top, bb = dh - x, dl = (x - (dh - bb)) - (top + bb), yh = dh * ch;
        if (!(yh > -150.f)) return 0.f;
        return exp2f(yh) * fmaf(fmaf(dh, ch, -yh) + fmaf(dh, cl, dl * ch), 0.693147182f, 1.f);
    }
};

template <typename T>
__device__ __forceinline__ float load(const void *row, int i) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(((const __nv_bfloat16 *)row)[i]);
    else return ((const float *)row)[i];
}

template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

struct Pair {
    u64 mass, count;
};
// Sums over the CTA, for every thread.
__device__ Pair block_sum(Pair v, Pair *s) {
    v.mass = warp_sum(v.mass), v.count = warp_sum(v.count);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
    for (int w = 1; w < kWarps; ++w) v.mass += s[w].mass, v.count += s[w].count;
    return v;
}

// A CTA a row. The cut is found by bisection over the values' keys.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample(SampleArgs a) {
    __shared__ Pair part[kWarps];
    __shared__ float top_s[kWarps];
    __shared__ int found_s;
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = a.V;
    pdl_wait();
    pdl_trigger();
    const void *row = (const char *)a.logits + (size_t)r * a.stride * sizeof(T);
    const float temp = a.temperature ? a.temperature[r] : 1.f, top_p = a.top_p ? a.top_p[r] : 1.f,
                min_p = a.min_p ? a.min_p[r] : 0.f, u = a.u ? a.u[r] : 0.f;
    const int top_k = a.top_k ? a.top_k[r] : 0;
    float top = -INFINITY;
    bool bad = false;
    for (int i = tid; i < V; i += kThreads) {
        const float x = load<T>(row, i);
        bad |= !(x < INFINITY);
        top = fmaxf(top, x);
    }
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    if (lane == 0) top_s[warp] = top;
    bad = __syncthreads_or(bad);
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, top_s[w]);
    bad |= top == -INFINITY;
    const bool wrong = !(temp >= 0.f && temp < INFINITY) || isnan(top_p) || isnan(min_p) || top_k < 0 || !(u >= 0.f && u < 1.f);
    if (bad || wrong) {
        if (tid == 0) flag(a.status, (bad ? TS_STATUS_NONFINITE : 0u) | (wrong ? TS_STATUS_INDEX : 0u));
        if (tid == 0 && a.token) a.token[r] = -1;
        for (int i = tid; i < V; i += kThreads) {
            if (a.probs) a.probs[(size_t)r * V + i] = NAN;
            if (a.kept) a.kept[(size_t)r * V + i] = NAN;
        }
        return;
    }
    const bool greedy = temp < 7.888609052210118e-31f;   // 2^-100
    const double c = 1.4426950408889634 / (greedy ? 1.0 : (double)temp);
    const Weights weight{top, (float)c, (float)(c - (double)(float)c)};

    // mass and count of the tokens of key lo or more
    auto from = [&](uint32_t lo, bool masses) {
        Pair v{0, 0};
        for (int i = tid; i < V; i += kThreads) {
            const float x = load<T>(row, i);
            if (key_of(x) >= lo) {
                ++v.count;
                if (masses) v.mass += weight(x);
            }
        }
        return block_sum(v, part);
    };
    const uint32_t key_top = key_of(top);
    uint32_t cut = kKeyLowest;   // key of the last token kept
    u64 ties = ~0ull;            // tokens kept of that key
    if (min_p > 0.f && !greedy)
        cut = max(cut, key_of(__double2float_ru((double)top + (double)temp * log((double)fminf(min_p, 1.f)))));
    if (greedy) cut = key_top, ties = 1;
    else if (top_k > 0 && from(cut, false).count > (u64)top_k) {
        uint32_t lo = cut, hi = key_top + 1;   // count(lo) >= k > count(hi)
        while (hi - lo > 1) {
            const uint32_t m = lo + (hi - lo) / 2;
            if (from(m, false).count >= (u64)top_k) lo = m;
            else hi = m;
        }
        cut = lo, ties = top_k - from(lo + 1, false).count;
    }
    Pair above = from(cut + 1, true), all = from(cut, false);
    u64 wt = cut <= key_top ? weight(value_of(cut)) : 0;
    ties = min(ties, all.count - above.count);
    if (top_p < 1.f && !greedy) {
        const u64 S = above.mass + ties * wt;
        // a token is kept where the mass before it is below this
        const u64 P = max(1ull, (u64)ceil((double)fmaxf(top_p, 0.f) * (double)S));
        if (above.mass >= P) {   // the cut is higher up
            uint32_t lo = cut, hi = key_top + 1;   // mass(lo) >= P > mass(hi), of whole values
            ++lo;
            while (hi - lo > 1) {
                const uint32_t m = lo + (hi - lo) / 2;
                if (from(m, true).mass >= P) lo = m;
                else hi = m;
            }
            cut = lo;
            above = from(cut + 1, true), all = from(cut, false);
            wt = weight(value_of(cut));
            ties = all.count - above.count;
        }
        ties = min(ties, wt ? (P - above.mass + wt - 1) / wt : ties);
    }
    // the id up to which tokens of the cut's key are kept: warps own ranges of ids
    const int per = (V + kWarps - 1) / kWarps, v0 = min(V, warp * per), v1 = min(V, v0 + per);
    auto before_warp = [&](u64 mine) {   // what the warps before this one hold
        __syncthreads();
        if (lane == 0) part[warp].mass = mine;
        __syncthreads();
        u64 s = 0;
        for (int w = 0; w < warp; ++w) s += part[w].mass;
        return s;
    };
    int id_cut = V;
    if (ties < all.count - above.count) {
        u64 n = 0;
        for (int i = v0 + lane; i < v1; i += 32) n += key_of(load<T>(row, i)) == cut;
        n = warp_sum(n);
        u64 at = before_warp(n);
        if (at < ties && ties <= at + n)
            for (int i0 = v0; i0 < v1; i0 += 32) {
                const unsigned is = __ballot_sync(~0u, i0 + lane < v1 && key_of(load<T>(row, min(i0 + lane, V - 1))) == cut);
                if (at < ties && at + __popc(is) >= ties) {
                    unsigned k = is;
                    for (u64 j = at + 1; j < ties; ++j) k &= k - 1;
                    if (lane == 0) found_s = i0 + __ffs(k) - 1;
                }
                at += __popc(is);
            }
        __syncthreads();
        id_cut = found_s;
    }
    auto kept = [&](float x, int i) { const uint32_t k = key_of(x); return k > cut || (k == cut && i <= id_cut); };
    const u64 S = above.mass + ties * wt;
    if (a.token) {
        // the first id at which the running sum is above u S; with none, the last of any mass
        const u64 want = min((u64)floor((double)u * (double)S), S - 1);
        u64 m = 0;
        for (int i = v0 + lane; i < v1; i += 32) {
            const float x = load<T>(row, i);
            if (kept(x, i)) m += weight(x);
        }
        m = warp_sum(m);
        u64 at = before_warp(m);
        if (at <= want && want < at + m)
            for (int i0 = v0; i0 < v1; i0 += 32) {
                const int i = i0 + lane;
                const float x = load<T>(row, min(i, V - 1));
                u64 w = i < v1 && kept(x, i) ? weight(x) : 0;
                for (int o = 1; o < 32; o <<= 1) {
                    const u64 y = __shfl_up_sync(~0u, w, o);
                    if (lane >= o) w += y;
                }
                const unsigned over = __ballot_sync(~0u, at + w > want);
                if (over) {
                    if (lane == 0) a.token[r] = i0 + __ffs(over) - 1;
                    break;
                }
                at += __shfl_sync(~0u, w, 31);
            }
    }
    if (a.probs || a.kept) {
        const float inv = (float)(1099511627776.0 / (double)S);
        __syncthreads();   // kept may be the logits
        for (int i = tid; i < V; i += kThreads) {
            const float x = load<T>(row, i);
            const bool k = kept(x, i);
            if (a.probs) a.probs[(size_t)r * V + i] = k ? weight.real(x) * inv : 0.f;
            if (a.kept) a.kept[(size_t)r * V + i] = k ? x : TS_DROPPED_LOGIT;
        }
    }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, ts_dtype dt, cudaStream_t s) {
    return dt == TS_BF16 ? launch(k_sample<__nv_bfloat16>, dim3(a.R), dim3(kThreads), 0, s, a)
                         : launch(k_sample<float>, dim3(a.R), dim3(kThreads), 0, s, a);
}

}  // namespace ts
