// kv8.cu -- head norms with rotation, and the 8-bit KV cache's append, read-back
// and commit.
//
// The cache is the shared tree cache of SpecInfer (arXiv 2305.09781, sec. 4.2)
// held as e4m3 codes with one fp32 scale per (row, head): node v of request b at
// row P_b + dfs(v), the accepted path's rows kept after verification.
#include "kv8.cuh"

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

// ---- norm, rotation, quantised append ---------------------------------------
struct RowArgs {
    const uint4 *q, *k, *v;              // node rows, *_stride 16-byte vectors apart
    long long q_stride, k_stride, v_stride;
    uint4 *q_out, *k_out;                // contiguous [B][n_max][H][d]; k_out without the cache
    int Hq, Hk, Hv;                      // heads handled here (0 leaves a projection out)
    const float *inv_freq, *q_weight, *k_weight;
    float eps;
    int norm, rot_dim, interleaved;
    ts_tree t;
    // append only
    uint8_t *k8, *v8;
    float *k_scale, *v_scale;
    const int32_t *prefix_len;
    int L_max;
    PagedArgs pg;
    uint32_t *status;
    int rows_per_cta;
};

constexpr int kRowThreads = 256;

// One CTA per (node, group of its heads). A row (one head's d values) is held
// by LPR = d / E lanes, E values of 16 bytes each, the same E positions of
// every row a lane meets, so the angles' cosines and sines and the norm weights
// stay in registers over the CTA's rows. The d / 2 angles are formed once per
// CTA: position times frequency and its remainder by 2 pi in fp64 (four
// operations an angle; an fp32 product at position 131072 is off by up to 4e-3),
// then sincosf of the fp32 remainder. Sums over a row are shuffles among its
// lanes. Memory bound: each element is read once and written once; kRowsAhead
// rows per lane group are loaded before any of them is worked on.
template <typename T, int D, bool APPEND>
__global__ void __launch_bounds__(kRowThreads) k_head_rows(RowArgs a) {
    constexpr int E = Vec<T>::E, LPR = D / E, RPC = kRowThreads / LPR, AHEAD = 2;
    __shared__ float2 cs_s[D / 2];
    __shared__ int bad_s;
    const int n_max = a.t.n_max, b = blockIdx.x / n_max, v = blockIdx.x - b * n_max;
    const int tid = threadIdx.x, sub = tid % LPR, slot = tid / LPR;
    const int e0 = sub * E;
    pdl_wait();
    pdl_trigger();
    const int n = a.t.n_nodes[b];
    const int dfs = a.t.dfs_of[(size_t)b * n_max + v];
    const int P = APPEND ? a.prefix_len[b] : 0;
    if (v >= n || dfs < 0 || dfs >= n_max) return;
    if (APPEND && (P < 0 || P > a.L_max - n)) {
        if (v == 0 && blockIdx.y == 0 && tid == 0) flag(a.status, TS_STATUS_INDEX);
        return;
    }
    const int rows = a.Hq + a.Hk + a.Hv;
    const int r_begin = blockIdx.y * a.rows_per_cta, r_end = min(rows, r_begin + a.rows_per_cta);
    const size_t node = (size_t)b * n_max + v;
    auto src = [&](int r) -> const uint4 * {
        if (r < a.Hq) return a.q + node * a.q_stride + (size_t)r * LPR + sub;
        r -= a.Hq;
        if (r < a.Hk) return a.k + node * a.k_stride + (size_t)r * LPR + sub;
        return a.v + node * a.v_stride + (size_t)(r - a.Hk) * LPR + sub;
    };
    // the first rows' loads are in flight while the angles are formed
    uint4 u[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (r_begin + slot + i * RPC < r_end) u[i] = __ldcs(src(r_begin + slot + i * RPC));
    if (APPEND) {
        if (tid == 0) bad_s = 0;
        __syncthreads();
        // a request with a page outside the table's range is skipped whole: every page of its rows P .. P + n - 1
        if (a.pg.bt && tid <= (P + n - 1) / TS_PAGE_KEYS - P / TS_PAGE_KEYS) {
            const int page = a.pg.bt[(size_t)b * a.pg.max_pages + P / TS_PAGE_KEYS + tid];
            if (page < 0 || page >= a.pg.num_pages) bad_s = 1;
        }
    }
    const int half = a.rot_dim >> 1;
    if (tid < half) {
        constexpr double kTwoPi = 6.283185307179586476925;
        const double ang = (double)a.t.pos[(size_t)b * n_max + dfs] * (double)a.inv_freq[tid];
        const float r = (float)fma(-kTwoPi, rint(ang * (1.0 / kTwoPi)), ang);
        float sn, c;
        sincosf(r, &sn, &c);
        cs_s[tid] = make_float2(c, sn);
    }
    __syncthreads();
    if (APPEND && bad_s) {
        if (v == 0 && blockIdx.y == 0 && tid == 0) flag(a.status, TS_STATUS_INDEX);
        return;
    }
    // y[e] = x[e] * ca[e] + partner * sa[e]; the partner of position p is p +- rot_dim/2
    // (the same slot of another lane) or, interleaved, the pair's other value
    float ca[E], sa[E];
    const bool turned = e0 < a.rot_dim;
    int partner = tid & 31;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        ca[e] = 1.f;
        sa[e] = 0.f;
        if (turned) {
            const int p = e0 + e;
            const bool low = a.interleaved ? !(p & 1) : p < half;
            const float2 cs = cs_s[a.interleaved ? p >> 1 : (low ? p : p - half)];
            ca[e] = cs.x;
            sa[e] = low ? -cs.y : cs.y;
        }
    }
    if (turned && !a.interleaved) partner += (e0 < half ? half : -half) / E;
    const unsigned group = LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u) << ((tid & 31) / LPR * LPR);

    long long row0 = 0, hs = 0;
    if (APPEND) {   // cache row of head 0; head h is h * hs rows further
        row0 = cache_row(a.pg, b, 0, a.Hv, a.L_max, P + dfs);
        hs = a.pg.bt ? TS_PAGE_KEYS : a.L_max;
    }
    for (int base = r_begin + slot; base < r_end; base += AHEAD * RPC) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int r = base + i * RPC;
            if (r >= r_end) break;
            const bool is_q = r < a.Hq, is_v = r >= a.Hq + a.Hk;
            float x[E];
            Vec<T>::unpack(u[i], x);
            if (!is_v) {
                if (a.norm) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                    for (int o = LPR / 2; o; o >>= 1) ss += __shfl_xor_sync(group, ss, o);
                    const float inv = rsqrtf(ss * (1.f / D) + a.eps);
                    const float *w = is_q ? a.q_weight : a.k_weight;
#pragma unroll
                    for (int e = 0; e < E; ++e) x[e] = x[e] * inv * (w ? __ldg(w + e0 + e) : 1.f);
                }
                if (half) {
                    float y[E];
                    if (a.interleaved) {
#pragma unroll
                        for (int e = 0; e < E; ++e) y[e] = x[e ^ 1];
                    } else {
#pragma unroll
                        for (int e = 0; e < E; ++e) y[e] = __shfl_sync(group, x[e], partner);
                    }
                    if (turned) {
#pragma unroll
                        for (int e = 0; e < E; ++e) x[e] = x[e] * ca[e] + y[e] * sa[e];
                    }
                }
            }
            if (is_q || !APPEND) {
                const int h = is_q ? r : r - a.Hq;
                uint4 *o = is_q ? a.q_out + (node * a.Hq + h) * LPR : a.k_out + (node * a.Hk + h) * LPR;
                o[sub] = Vec<T>::pack(x);
            } else {
                const int h = is_v ? r - a.Hq - a.Hk : r - a.Hq;
                float top = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) top = max_nan(top, fabsf(x[e]));
#pragma unroll
                for (int o = LPR / 2; o; o >>= 1) top = max_nan(top, __shfl_xor_sync(group, top, o));
                const bool fine = top <= 3.402823466e38f;   // false for infinities and NaN
                const float scale = fmaxf(__fdiv_rn(top, kFp8Max), kScaleMin);
                const float inv = __fdiv_rn(1.f, scale);
                uint32_t c[E / 4];
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(x[e], inv), __fmul_rn(x[e + 1], inv)),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(x[e + 2], inv), __fmul_rn(x[e + 3], inv)),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    c[e / 4] = fine ? lo | hi << 16 : 0u;
                }
                const size_t row = (size_t)(row0 + h * hs);
                uint8_t *dst = (is_v ? a.v8 : a.k8) + row * D + e0;
                if constexpr (E == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0], c[1]);
                else *reinterpret_cast<uint32_t *>(dst) = c[0];
                if (sub == 0) {
                    (is_v ? a.v_scale : a.k_scale)[row] = fine ? scale : __int_as_float(0x7fc00000);
                    if (!fine) flag(a.status, TS_STATUS_NONFINITE);
                }
            }
            const int nr = r + AHEAD * RPC;   // this slot's next row
            if (nr < r_end) u[i] = __ldcs(src(nr));
        }
    }
}

template <typename T, int D, bool APPEND>
cudaError_t rows_launch(RowArgs &a, cudaStream_t s) {
    constexpr int RPC = kRowThreads / (D / Vec<T>::E);
    const int rows = a.Hq + a.Hk + a.Hv;
    const long long nodes = (long long)a.t.B * a.t.n_max;
    // heads of a node are split over CTAs only while that gives each SM more to do
    long long groups = 2LL * num_sms() / nodes;
    const int most = (rows + RPC - 1) / RPC;
    if (groups > most) groups = most;
    if (groups < 1) groups = 1;
    a.rows_per_cta = ((rows + (int)groups - 1) / (int)groups + RPC - 1) / RPC * RPC;
    const dim3 grid((unsigned)nodes, (rows + a.rows_per_cta - 1) / a.rows_per_cta);
    return launch(k_head_rows<T, D, APPEND>, grid, dim3(kRowThreads), 0, s, a);
}

template <bool APPEND>
cudaError_t rows_dispatch(RowArgs &a, int d, ts_dtype dt, cudaStream_t s) {
    if (dt == TS_BF16)
        return d == 128 ? rows_launch<__nv_bfloat16, 128, APPEND>(a, s) : rows_launch<__nv_bfloat16, 64, APPEND>(a, s);
    return d == 128 ? rows_launch<float, 128, APPEND>(a, s) : rows_launch<float, 64, APPEND>(a, s);
}

void set_rope(RowArgs &a, const ts_qk_rope &r) {
    a.inv_freq = r.inv_freq;
    a.q_weight = r.q_weight;
    a.k_weight = r.k_weight;
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
// Memory bound: d + 4 bytes in, d * sizeof(T) out a row.
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
// depth), so rounds need no order among themselves beyond that.
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
    const int per = 16 / (dt == TS_BF16 ? 2 : 4);
    RowArgs a = {};
    a.q = (const uint4 *)q;
    a.k = (const uint4 *)k;
    a.q_stride = q_stride / per;
    a.k_stride = k_stride / per;
    a.q_out = (uint4 *)q_out;
    a.k_out = (uint4 *)k_out;
    a.Hq = Hq;
    a.Hk = Hk;
    set_rope(a, rope);
    a.t = t;
    return rows_dispatch<false>(a, d, dt, s);
}

cudaError_t launch_kv8_append(const ts_kv8 &kv, const void *k_new, const void *v_new, long long k_stride,
                              long long v_stride, const ts_qk_rope *rope, void *q_out, const void *q, int Hq,
                              long long q_stride, const int32_t *prefix_len, const ts_tree &t, ts_dtype dt,
                              uint32_t *status, cudaStream_t s) {
    const int per = 16 / (dt == TS_BF16 ? 2 : 4);
    RowArgs a = {};
    a.q = (const uint4 *)q;
    a.k = (const uint4 *)k_new;
    a.v = (const uint4 *)v_new;
    a.q_stride = q_stride / per;
    a.k_stride = k_stride / per;
    a.v_stride = v_stride / per;
    a.q_out = (uint4 *)q_out;
    a.Hq = Hq;
    a.Hk = kv.H;
    a.Hv = kv.H;
    if (rope) set_rope(a, *rope);
    a.t = t;
    a.k8 = kv.k;
    a.v8 = kv.v;
    a.k_scale = kv.k_scale;
    a.v_scale = kv.v_scale;
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
