// kv8.cu -- head norms with rotation, and the 8-bit KV cache's append, read-back
// and commit.
//
// The cache is the shared tree cache of SpecInfer (arXiv 2305.09781, sec. 4.2)
// held as e4m3 codes with one fp32 scale per (row, head): node v of request b at
// row P_b + dfs(v), the accepted path's rows kept after verification.
#include "kv8.cuh"

#include <algorithm>
#include <type_traits>

namespace ts {
namespace {

// ---- elements of a row, 16 bytes at a time ----------------------------------
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int E = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec<float> {
    static constexpr int E = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

// Maximum that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Largest magnitude of three, a NaN kept.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float y;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ---- norm, rotation, quantised append ---------------------------------------
struct RowArgs {
    // by projection: queries, keys, values (0 heads leave one out)
    const void *src[3];                  // node rows, stride values from one node to the next
    long long stride[3];
    int heads[3], groups[3], per_group[3];   // CTAs a node and heads in each, set by rows_launch
    void *out[2];                        // contiguous [B][n_max][H][d]; keys only without the cache
    const float *weight[2];
    const float *inv_freq;
    float eps;
    int norm, rot_dim, interleaved;
    ts_tree t;
    // append only, keys and values
    uint8_t *codes[2];
    float *scales[2];
    const int32_t *prefix_len;
    int L_max;
    PagedArgs pg;
    uint32_t *status;
};

constexpr int kRowThreads = 128, kRowPasses = 8;   // rows of a CTA: kRowPasses a lane group, 16 KB

// Two values of a row as one 4-byte (bf16) or 8-byte (fp32) piece.
template <typename T>
struct Two;
template <>
struct Two<__nv_bfloat16> {
    using U = uint32_t;
    static __device__ __forceinline__ float2 get(U u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    static __device__ __forceinline__ U put(float2 x) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x.x, x.y);
        return *reinterpret_cast<const U *>(&p);
    }
};
template <>
struct Two<float> {
    using U = uint2;
    static __device__ __forceinline__ float2 get(U u) { return make_float2(__uint_as_float(u.x), __uint_as_float(u.y)); }
    static __device__ __forceinline__ U put(float2 x) { return make_uint2(__float_as_uint(x.x), __float_as_uint(x.y)); }
};

// Values t (as they lie: the lane's first piece, then its second) as H rotation pairs (x, y), two pairs a vector, and back.
template <int H, bool INTER>
__device__ __forceinline__ void pairs(const float2 (&t)[H], float2 (&x)[H / 2], float2 (&y)[H / 2]) {
#pragma unroll
    for (int e = 0; e < H / 2; ++e) {
        x[e] = INTER ? make_float2(t[2 * e].x, t[2 * e + 1].x) : t[e];
        y[e] = INTER ? make_float2(t[2 * e].y, t[2 * e + 1].y) : t[H / 2 + e];
    }
}
template <int H, bool INTER>
__device__ __forceinline__ void unpairs(const float2 (&x)[H / 2], const float2 (&y)[H / 2], float2 (&t)[H]) {
#pragma unroll
    for (int e = 0; e < H / 2; ++e) {
        t[INTER ? 2 * e : e] = INTER ? make_float2(x[e].x, y[e].x) : x[e];
        t[INTER ? 2 * e + 1 : H / 2 + e] = INTER ? make_float2(x[e].y, y[e].y) : y[e];
    }
}

// One CTA per (node, projection, group of its heads). A row (one head's d
// values) is held by LPR lanes, E = d / LPR values each in two pieces of 8
// bytes: the first members of E / 2 rotation pairs and the second ones
// (interleaved pairs: 16 bytes in a row), so a rotation needs no other lane; a
// row's only shuffles are those of its sum of squares (and, quantised, of its
// largest value). The lane's cosines, sines and norm weights stay in registers
// over the CTA's rows. The angles are formed once per CTA: position times
// frequency and its remainder by 2 pi in fp64 (an fp32 product at position
// 131072 is off by up to 4e-3), then sincosf of the fp32 remainder. Each value
// is read once and written once, all of a CTA's rows in flight from its start
// (into shared memory; in registers, four rows a lane group ahead, they cost
// more occupancy than they hid: 51 us against 46 on an append of 64 x 47 nodes,
// 56 + 56 heads of 128). What bounds a large call next to memory is issuing
// (67% of the slots in that append): the loop is compiled once for each kind of
// row (query, key, value), and a CTA runs one of them; one loop for all kinds
// took 56 us. Measured there: norm and rotation of q and k 30.1 us (172 MB, 84%
// of the copy peak), the append with its codes 45.3 us (217 MB, 71%). The
// divisions are the definition's and cost 1.6 us of that.
template <typename T, int D, bool APPEND, bool INTER>
__global__ void __launch_bounds__(kRowThreads) k_head_rows(RowArgs a) {
    constexpr int E = 16 / (int)sizeof(T), LPR = D / E, RPC = kRowThreads / LPR, RW = 32 / LPR, H = E / 2;
    constexpr int ROW = D * (int)sizeof(T);   // bytes
    __shared__ __align__(16) uint8_t rows_s[kRowPasses * RPC * ROW];
    __shared__ float2 cs_s[D / 2];
    __shared__ int bad_s;
    const int n_max = a.t.n_max, b = blockIdx.x / n_max, dfs = blockIdx.x - b * n_max;
    const int tid = threadIdx.x, sub = tid % LPR, slot = tid / LPR;
    const int half = a.rot_dim >> 1;
    const int kind = (int)blockIdx.y < a.groups[0] ? 0 : (int)blockIdx.y < a.groups[0] + a.groups[1] ? 1 : 2;
    // this lane's pairs p0 .. p0 + H - 1: pair p is (p, p + half), or behind the rotated part (unrotated) the
    // same with that part's halves
    const int p0 = sub * H;
    const bool turned = p0 < half;
    const int e0 = INTER ? 2 * p0 : turned ? p0 : p0 + half;
    const int e1 = INTER ? e0 + H : turned ? p0 + half : p0 + D / 2;
    pdl_wait();
    pdl_trigger();
    const int n = a.t.n_nodes[b];
    const int v = a.t.perm[blockIdx.x];   // of nodes past the last, too: no load waits for another
    const int pos = kind < 2 && half ? a.t.pos[blockIdx.x] : 0;
    const int P = APPEND ? a.prefix_len[b] : 0;
    if (dfs >= n || v < 0 || v >= n_max) return;
    if (APPEND && (P < 0 || P > a.L_max - n)) {
        if (dfs == 0 && blockIdx.y == 0 && tid == 0) flag(a.status, TS_STATUS_INDEX);
        return;
    }
    const int part = blockIdx.y - (kind == 0 ? 0 : kind == 1 ? a.groups[0] : a.groups[0] + a.groups[1]);
    const int r_begin = part * a.per_group[kind], r_end = min(a.heads[kind], r_begin + a.per_group[kind]);
    const size_t node = (size_t)b * n_max + v;
    const T *src = (const T *)a.src[kind] + node * a.stride[kind] + (size_t)(r_begin + slot) * D + sub * E;
    uint8_t *mine = rows_s + slot * ROW;
#pragma unroll
    for (int i = 0; i < kRowPasses; ++i)
        if (r_begin + slot + i * RPC < r_end) cp_async16(mine + i * RPC * ROW + sub * 16, src + i * RPC * D);
    if (APPEND) {
        if (tid == 0) bad_s = 0;
        __syncthreads();
        // a request with a page outside the table's range is skipped whole: every page of its rows P .. P + n - 1
        if (a.pg.bt && tid <= (P + n - 1) / TS_PAGE_KEYS - P / TS_PAGE_KEYS) {
            const int page = a.pg.bt[(size_t)b * a.pg.max_pages + P / TS_PAGE_KEYS + tid];
            if (page < 0 || page >= a.pg.num_pages) bad_s = 1;
        }
    }
    if (tid < half && kind < 2) {
        constexpr double kTwoPi = 6.283185307179586476925;
        const double ang = (double)pos * (double)a.inv_freq[tid];
        const float r = (float)fma(-kTwoPi, rint(ang * (1.0 / kTwoPi)), ang);
        float sn, c;
        sincosf(r, &sn, &c);
        cs_s[tid] = make_float2(c, sn);
    }
    cp_async_wait_all();
    __syncthreads();
    if (APPEND && bad_s) {
        if (dfs == 0 && blockIdx.y == 0 && tid == 0) flag(a.status, TS_STATUS_INDEX);
        return;
    }
    auto rows = [&](auto kind_c) {
        constexpr int KIND = decltype(kind_c)::value;
        constexpr bool TURN = KIND < 2, QUANT = APPEND && KIND > 0;
        // weights and rotation of the lane's pairs (p, q), two pairs a vector:
        // p -> inv * (p * pc + q * qs), q -> inv * (q * qc + p * ps)
        float2 pc[H / 2], qs[H / 2], qc[H / 2], ps[H / 2];
        if constexpr (TURN) {
            const float *wp = a.weight[KIND];
            float w[4][H];
#pragma unroll
            for (int e = 0; e < H; ++e) {
                const float2 c = turned ? cs_s[p0 + e] : make_float2(1.f, 0.f);
                const float wx = wp ? __ldg(wp + (INTER ? e0 + 2 * e : e0 + e)) : 1.f;
                const float wy = wp ? __ldg(wp + (INTER ? e0 + 2 * e + 1 : e1 + e)) : 1.f;
                w[0][e] = wx * c.x;
                w[1][e] = -wy * c.y;
                w[2][e] = wy * c.x;
                w[3][e] = wx * c.y;
            }
#pragma unroll
            for (int e = 0; e < H / 2; ++e) {
                pc[e] = make_float2(w[0][2 * e], w[0][2 * e + 1]);
                qs[e] = make_float2(w[1][2 * e], w[1][2 * e + 1]);
                qc[e] = make_float2(w[2][2 * e], w[2][2 * e + 1]);
                ps[e] = make_float2(w[3][2 * e], w[3][2 * e + 1]);
            }
        }
        // where the lane group's first row goes: values, or codes and a scale
        T *out = nullptr;
        uint8_t *codes = nullptr;
        float *scales = nullptr;
        long long hs = 0;   // cache rows from one head to the next
        if constexpr (QUANT) {
            const long long row = cache_row(a.pg, b, r_begin + slot, a.heads[KIND], a.L_max, P + dfs);
            hs = a.pg.bt ? TS_PAGE_KEYS : a.L_max;
            codes = a.codes[KIND - 1] + (size_t)row * D;
            scales = a.scales[KIND - 1] + row;
        } else {
            out = (T *)a.out[KIND] + (node * a.heads[KIND] + r_begin + slot) * D;
        }
        // the rows of a warp's lane groups go together (none of them leaves early), so every shuffle is the whole warp's
        const T *in = reinterpret_cast<const T *>(mine);
        // r: this group's row, first: the warp's first
#pragma unroll 1
        for (int r = r_begin + slot, first = r_begin + slot / RW * RW; first < r_end; r += RPC, first += RPC) {
            float2 t[H];
            const uint2 lo = *reinterpret_cast<const uint2 *>(in + e0), hi = *reinterpret_cast<const uint2 *>(in + e1);
            in += RPC * D;
            if constexpr (sizeof(T) == 2) {
                t[0] = Two<T>::get(lo.x);
                t[1] = Two<T>::get(lo.y);
                t[2] = Two<T>::get(hi.x);
                t[3] = Two<T>::get(hi.y);
            } else {
                t[0] = Two<T>::get(lo);
                t[1] = Two<T>::get(hi);
            }
            if (TURN && (a.norm || half)) {
                float2 x[H / 2], y[H / 2];   // first and second members
                pairs<H, INTER>(t, x, y);
                if (a.norm) {
                    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
                    for (int e = 0; e < H / 2; ++e) s2 = __ffma2_rn(y[e], y[e], __ffma2_rn(x[e], x[e], s2));
                    float ss = s2.x + s2.y;
#pragma unroll
                    for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
                    const float inv = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
                    for (int e = 0; e < H / 2; ++e) {
                        x[e] = __fmul2_rn(x[e], make_float2(inv, inv));
                        y[e] = __fmul2_rn(y[e], make_float2(inv, inv));
                    }
                }
#pragma unroll
                for (int e = 0; e < H / 2; ++e) {
                    const float2 p = x[e], q = y[e];
                    x[e] = __fmul2_rn(p, pc[e]);
                    y[e] = __fmul2_rn(q, qc[e]);
                    if (turned) {   // an unrotated pair's members keep apart, an infinity in one of them too
                        x[e] = __ffma2_rn(q, qs[e], x[e]);
                        y[e] = __ffma2_rn(p, ps[e], y[e]);
                    }
                }
                unpairs<H, INTER>(x, y, t);
            }
            if constexpr (QUANT) {
                float top = 0.f;
#pragma unroll
                for (int e = 0; e < H; ++e) top = max_abs(top, t[e].x, t[e].y);
#pragma unroll
                for (int o = LPR / 2; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(~0u, top, o));
                if (r < r_end) {
                    const bool fine = top <= 3.402823466e38f;   // false for infinities and NaN
                    const float scale = fmaxf(__fdiv_rn(top, kFp8Max), kScaleMin);
                    const float rs = __frcp_rn(scale);
                    uint32_t c[H];   // two codes each
#pragma unroll
                    for (int e = 0; e < H; ++e)
                        c[e] = __nv_cvt_float2_to_fp8x2(__fmul2_rn(t[e], make_float2(rs, rs)), __NV_SATFINITE, __NV_E4M3);
                    if constexpr (sizeof(T) == 2) {
                        *reinterpret_cast<uint32_t *>(codes + e0) = fine ? c[0] | c[1] << 16 : 0u;
                        *reinterpret_cast<uint32_t *>(codes + e1) = fine ? c[2] | c[3] << 16 : 0u;
                    } else {
                        *reinterpret_cast<uint16_t *>(codes + e0) = (uint16_t)(fine ? c[0] : 0u);
                        *reinterpret_cast<uint16_t *>(codes + e1) = (uint16_t)(fine ? c[1] : 0u);
                    }
                    if (sub == 0) {
                        *scales = fine ? scale : __int_as_float(0x7fc00000);
                        if (!fine) flag(a.status, TS_STATUS_NONFINITE);
                    }
                }
                codes += RPC * hs * D;
                scales += RPC * hs;
            } else {
                if (r < r_end) {
                    uint2 lo, hi;
                    if constexpr (sizeof(T) == 2) {
                        lo = make_uint2(Two<T>::put(t[0]), Two<T>::put(t[1]));
                        hi = make_uint2(Two<T>::put(t[2]), Two<T>::put(t[3]));
                    } else {
                        lo = Two<T>::put(t[0]);
                        hi = Two<T>::put(t[1]);
                    }
                    *reinterpret_cast<uint2 *>(out + e0) = lo;
                    *reinterpret_cast<uint2 *>(out + e1) = hi;
                }
                out += RPC * D;
            }
        }
    };
    if (kind == 0) rows(std::integral_constant<int, 0>());
    else if (kind == 1) rows(std::integral_constant<int, 1>());
    else if constexpr (APPEND) rows(std::integral_constant<int, 2>());
}

template <typename T, int D, bool APPEND>
cudaError_t rows_launch(RowArgs &a, cudaStream_t s) {
    constexpr int RPC = kRowThreads / (D * (int)sizeof(T) / 16);
    const long long nodes = (long long)a.t.B * a.t.n_max;
    // a projection's heads are split over CTAs only while that gives each SM more to do
    int ctas = 0;
    for (int i = 0; i < 3; ++i) {
        if (!a.heads[i]) continue;   // left out: no groups
        const int most = (a.heads[i] + RPC - 1) / RPC;
        const int least = (most + kRowPasses - 1) / kRowPasses;
        const int groups = (int)std::max<long long>(least, std::min<long long>(most, num_sms() / nodes));
        a.per_group[i] = ((a.heads[i] + groups - 1) / groups + RPC - 1) / RPC * RPC;
        a.groups[i] = (a.heads[i] + a.per_group[i] - 1) / a.per_group[i];
        ctas += a.groups[i];
    }
    const dim3 grid((unsigned)nodes, ctas);
    if (a.interleaved) return launch(k_head_rows<T, D, APPEND, true>, grid, dim3(kRowThreads), 0, s, a);
    return launch(k_head_rows<T, D, APPEND, false>, grid, dim3(kRowThreads), 0, s, a);
}

template <bool APPEND>
cudaError_t rows_dispatch(RowArgs &a, int d, ts_dtype dt, cudaStream_t s) {
    if (dt == TS_BF16)
        return d == 128 ? rows_launch<__nv_bfloat16, 128, APPEND>(a, s) : rows_launch<__nv_bfloat16, 64, APPEND>(a, s);
    return d == 128 ? rows_launch<float, 128, APPEND>(a, s) : rows_launch<float, 64, APPEND>(a, s);
}

void set_rope(RowArgs &a, const ts_qk_rope &r) {
    a.inv_freq = r.inv_freq;
    a.weight[0] = r.norm ? r.q_weight : nullptr;   // the weights are the norm's
    a.weight[1] = r.norm ? r.k_weight : nullptr;
    a.eps = r.eps;
    a.norm = r.norm != 0;
    a.rot_dim = r.rot_dim;
    a.interleaved = r.interleaved != 0;
}

// ---- read-back --------------------------------------------------------------
struct ReadArgs {
    uint4 *k_out, *v_out;
    const uint8_t *k8, *v8;
    const float *k_scale, *v_scale;
    const int32_t *row_begin, *row_end;
    int H, rows, L_out;
    PagedArgs pg;
    uint32_t *status;
};

constexpr int kReadThreads = 256, kReadRows = 64;

// One CTA per (64 output rows, head, request): a lane turns E codes (8 for
// bf16, 4 for fp32) into 16 bytes, so that both sides of the copy are
// contiguous over a warp; the CTA's loads are issued before its stores.
// Memory bound: d + 4 bytes in, d * sizeof(T) out a row; 16 requests of 512 to
// 4096 rows, 32 heads of 128, into bf16: 142 us, 98% of the copy peak.
template <typename T, int D>
__global__ void __launch_bounds__(kReadThreads) k_kv8_read(ReadArgs a) {
    constexpr int E = Vec<T>::E, LPR = D / E, RPC = kReadThreads / LPR, U = kReadRows / RPC;
    const int b = blockIdx.z, h = blockIdx.y, sub = threadIdx.x % LPR, slot = threadIdx.x / LPR;
    pdl_wait();
    pdl_trigger();
    const int begin = a.row_begin ? a.row_begin[b] : 0, end = a.row_end[b];
    if (begin < 0 || end < begin || end > a.rows || end - begin > a.L_out) {
        if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) flag(a.status, TS_STATUS_INDEX);
        return;
    }
    const int count = end - begin, j0 = blockIdx.x * kReadRows + slot;
    if ((int)blockIdx.x * kReadRows >= count) return;
    auto half = [&](const uint8_t *codes, const float *scales, uint4 *out) {
        uint2 c[U];
        float sc[U];
        bool has[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int j = j0 + i * RPC;
            has[i] = false;
            if (j < count) {
                const long long row = cache_row(a.pg, b, h, a.H, a.rows, begin + j);
                if (row < 0) {
                    flag(a.status, TS_STATUS_INDEX);
                } else {
                    has[i] = true;
                    const uint8_t *p = codes + (size_t)row * D + sub * E;
                    if constexpr (E == 8) c[i] = __ldcs(reinterpret_cast<const uint2 *>(p));
                    else c[i] = make_uint2(__ldcs(reinterpret_cast<const uint32_t *>(p)), 0u);
                    sc[i] = __ldg(scales + row);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (has[i]) {
                float x[E];
                const uint32_t w[2] = {c[i].x, c[i].y};
#pragma unroll
                for (int e = 0; e < E; e += 2) {
                    const float2 f = fp8x2_to_float2((uint16_t)(w[e / 4] >> (e % 4 * 8)));
                    x[e] = f.x * sc[i];
                    x[e + 1] = f.y * sc[i];
                }
                __stcs(out + (((size_t)b * gridDim.y + h) * a.L_out + j0 + i * RPC) * LPR + sub, Vec<T>::pack(x));
            }
    };
    half(a.k8, a.k_scale, a.k_out);
    half(a.v8, a.v_scale, a.v_out);
}

// ---- commit -----------------------------------------------------------------
// As k_kv_commit: one CTA per (request, group of heads); path node i moves from
// row P + dfs(path[i]) to row P + i in rounds of increasing i, each round
// reading all its pieces before any is written. A round's destinations are
// never a later round's sources (a node's depth-first index is at least its
// depth), so rounds need no order among themselves beyond that. Bound by the
// launch and one chain of loads: 2.9 us for 64 requests of 56 heads.
constexpr int kCommit8Threads = 256, kCommit8Heads = 8;

template <int D>
__global__ void __launch_bounds__(kCommit8Threads) k_kv8_commit(uint4 *k8, uint4 *v8, float *k_scale, float *v_scale,
                                                                const int32_t *prefix_len, int32_t *new_prefix_len,
                                                                const int32_t *out_path, const int32_t *out_count,
                                                                ts_tree t, int H, int rows, uint32_t *status,
                                                                PagedArgs pg) {
    constexpr int VPR = D / 16;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int h0 = blockIdx.y * kCommit8Heads, hn = min(H - h0, kCommit8Heads);
    const bool lead = blockIdx.y == 0;
    pdl_wait();
    pdl_trigger();
    __shared__ int dfs_s[kMaxNodes], src_s[kMaxNodes];
    __shared__ long long from_s[kMaxNodes], to_s[kMaxNodes];   // cache rows of head 0
    __shared__ int bad_s;
    static_assert(kCommit8Threads >= kMaxNodes, "a thread per path entry and per node");
    const int n = t.n_nodes[b], P = prefix_len[b], cnt = out_count[b];
    const int node = tid < t.n_max ? out_path[(size_t)b * (t.n_max + 1) + tid] : -1;
    const int dfs = tid < t.n_max ? t.dfs_of[(size_t)b * t.n_max + tid] : -1;
    if (tid == 0) bad_s = !(n > 0 && n <= t.n_max && cnt >= 0 && cnt <= n && P >= 0 && P <= rows - n);
    if (tid < t.n_max) dfs_s[tid] = dfs;
    __syncthreads();
    if (!bad_s && tid < cnt) {
        const int s = node >= 0 && node < n ? dfs_s[node] : -1;
        // a path node at depth i has a depth-first index of at least i
        if (s < tid || s >= n) {
            bad_s = 1;
        } else {
            src_s[tid] = s;
            from_s[tid] = cache_row(pg, b, 0, H, rows, P + s);
            to_s[tid] = cache_row(pg, b, 0, H, rows, P + tid);
            if (from_s[tid] < 0 || to_s[tid] < 0) bad_s = 1;
        }
    }
    __syncthreads();
    if (bad_s) {
        if (tid == 0 && lead) {
            if (cnt != 0 || (n > 0 && (P < 0 || P > rows - n))) flag(status, TS_STATUS_INDEX);
            new_prefix_len[b] = P;
        }
        return;
    }
    const long long hs = pg.bt ? TS_PAGE_KEYS : rows;
    const int per_i = hn * VPR, total = cnt * per_i;
    for (int r0 = 0; r0 < total; r0 += kCommit8Threads) {
        const int idx = r0 + tid, i = idx / per_i, rem = idx - i * per_i, h = h0 + rem / VPR, c = rem % VPR;
        const bool mv = idx < total && src_s[i] != i;
        uint4 kx, vx;
        float ks, vs;
        if (mv) {
            const size_t row = (size_t)(from_s[i] + h * hs);
            kx = k8[row * VPR + c];
            vx = v8[row * VPR + c];
            if (c == 0) {
                ks = k_scale[row];
                vs = v_scale[row];
            }
        }
        __syncthreads();
        if (mv) {
            const size_t row = (size_t)(to_s[i] + h * hs);
            k8[row * VPR + c] = kx;
            v8[row * VPR + c] = vx;
            if (c == 0) {
                k_scale[row] = ks;
                v_scale[row] = vs;
            }
        }
        __syncthreads();
    }
    if (tid == 0 && lead) new_prefix_len[b] = P + cnt;
}

}  // namespace

cudaError_t launch_qk_norm_rope(void *q_out, void *k_out, const void *q, const void *k, int Hq, int Hk, int d,
                                long long q_stride, long long k_stride, const ts_qk_rope &rope, const ts_tree &t,
                                ts_dtype dt, cudaStream_t s) {
    RowArgs a = {};
    a.src[0] = q;
    a.src[1] = k;
    a.stride[0] = q_stride;
    a.stride[1] = k_stride;
    a.out[0] = q_out;
    a.out[1] = k_out;
    a.heads[0] = Hq;
    a.heads[1] = Hk;
    set_rope(a, rope);
    a.t = t;
    return rows_dispatch<false>(a, d, dt, s);
}

cudaError_t launch_kv8_append(const ts_kv8 &kv, const void *k_new, const void *v_new, long long k_stride,
                              long long v_stride, const ts_qk_rope *rope, void *q_out, const void *q, int Hq,
                              long long q_stride, const int32_t *prefix_len, const ts_tree &t, ts_dtype dt,
                              uint32_t *status, cudaStream_t s) {
    RowArgs a = {};
    a.src[0] = q;
    a.src[1] = k_new;
    a.src[2] = v_new;
    a.stride[0] = q_stride;
    a.stride[1] = k_stride;
    a.stride[2] = v_stride;
    a.out[0] = q_out;
    a.heads[0] = Hq;
    a.heads[1] = a.heads[2] = kv.H;
    if (rope) set_rope(a, *rope);
    a.t = t;
    a.codes[0] = kv.k;
    a.codes[1] = kv.v;
    a.scales[0] = kv.k_scale;
    a.scales[1] = kv.v_scale;
    a.prefix_len = prefix_len;
    a.L_max = kv8_rows(kv);
    a.pg = kv8_pages(kv);
    a.status = status;
    return rows_dispatch<true>(a, kv.d, dt, s);
}

cudaError_t launch_kv8_read(void *k_out, void *v_out, const ts_kv8 &kv, const int32_t *row_begin,
                            const int32_t *row_end, int L_out, ts_dtype dt, uint32_t *status, cudaStream_t s) {
    ReadArgs a = {(uint4 *)k_out, (uint4 *)v_out, kv.k, kv.v, kv.k_scale, kv.v_scale, row_begin, row_end,
                  kv.H, kv8_rows(kv), L_out, kv8_pages(kv), status};
    const dim3 grid((L_out + kReadRows - 1) / kReadRows, kv.H, kv.B), block(kReadThreads);
    if (dt == TS_BF16)
        return kv.d == 128 ? launch(k_kv8_read<__nv_bfloat16, 128>, grid, block, 0, s, a)
                           : launch(k_kv8_read<__nv_bfloat16, 64>, grid, block, 0, s, a);
    return kv.d == 128 ? launch(k_kv8_read<float, 128>, grid, block, 0, s, a)
                       : launch(k_kv8_read<float, 64>, grid, block, 0, s, a);
}

cudaError_t launch_kv8_commit(const ts_kv8 &kv, const int32_t *prefix_len, int32_t *new_prefix_len,
                              const int32_t *out_path, const int32_t *out_count, const ts_tree &t, uint32_t *status,
                              cudaStream_t s) {
    const dim3 grid(t.B, (kv.H + kCommit8Heads - 1) / kCommit8Heads), block(kCommit8Threads);
    if (kv.d == 128)
        return launch(k_kv8_commit<128>, grid, block, 0, s, (uint4 *)kv.k, (uint4 *)kv.v, kv.k_scale, kv.v_scale,
                      prefix_len, new_prefix_len, out_path, out_count, t, kv.H, kv8_rows(kv), status, kv8_pages(kv));
    return launch(k_kv8_commit<64>, grid, block, 0, s, (uint4 *)kv.k, (uint4 *)kv.v, kv.k_scale, kv.v_scale,
                  prefix_len, new_prefix_len, out_path, out_count, t, kv.H, kv8_rows(kv), status, kv8_pages(kv));
}

}  // namespace ts
