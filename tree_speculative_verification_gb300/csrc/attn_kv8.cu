// attn_kv8.cu -- tree attention over the 8-bit KV cache, on tcgen05.
//
// TreeAttention(u) = Attention(S_u) for every node u of the token tree
// (SpecInfer, arXiv 2305.09781, Def. 4.1, Eq. 1-4; the mask of sec. 4.2), with
// K and V held as e4m3 codes times one fp32 scale per (row, head), and G query
// heads to a key/value head. The R = n * G query rows of a (request, key/value
// head) share its keys; they are taken in blocks of RP = 16, 32, 48 or 64.
//
// The cache's codes go to the tensor cores as they are. Both products are
// transposed, so that keys, then value dims, are the 128 rows of the MMA and a
// tile costs in proportion to the query rows there are:
//   S^T [128 keys x RP]    = K [128 x d] * Qh^T + K * Ql^T            (e4m3 * e4m3)
//   O^T [d x 3 RP]        += V^T [d x 128 keys] * [P0 | P1 | P2]^T (e4m3 * e5m2)
// What is not in 8 bits is split into several 8-bit numbers:
//   a query row, scaled by a power of two to a largest value in [128, 256), is
//   qh + ql with qh = e4m3(q), ql = e4m3(q - qh): bf16's eight bits exactly for
//   values down to 2^-10 of the row's largest, 2^-18 of it absolutely below;
//   a weight w = probability * value scale (2^7 at the reference) is rounded to
//   fp16, whose upper byte is an e5m2 number: w0 = upper byte of w, w1 = of
//   w - w0, w2 = of the rest, rounded. Nine bits down to 2^-15 of the weight at
//   the reference, to 2^-24 of it absolutely below (a pair of e4m3 numbers would
//   end at 2^-18: a long cache with one dominant key has weights there by the
//   thousand).
// Softmax: y = S * key scale * query scale is the exponent. What has to fit w's few
// bits is e^y times the value scale, so the running maximum of a query row is that
// of y + log2(value scale) over the keys the row sees: a large value that it does
// not see, or that has no weight, takes no bits from the others. The sums are of
// the probability alone, which then spans 2^-112 to 2^115 over the scales there
// are; factors between two references are applied as their root, twice. Sums,
// maxima, O: fp32.
//
// One CTA per SM takes units (request, head, RP query rows, range of tiles) from
// a queue in the workspace, longest first; ranges are cut only as far as the
// launch needs to fill the SMs, the last CTA of a cut item joining the parts.
//   warp 0      producer: K and V tiles by TMA into a ring of stages; the tile's
//               scales and, for tree keys, subtree ends by cp.async on the same
//               mbarrier
//   warp 1      issues the scores, as soon as a tile's buffer has been read
//   warp 2      issues O += P V
//   warp 3      takes units, publishes them in a ring of four, copies the next
//               unit's query rows into the other Q buffer
//   softmax     groups of four warps, lane = key, 8 or 16 columns (query rows) a
//               group. The reference maximum of a column is raised only when a
//               score passes it by 2^8 (one vote per tile and group), so the
//               common tile has no reduction over keys. Tree node j is seen by
//               the rows of its subtree, one interval of rows.
//   last four   split a unit's query rows in place, then write the unit before
//               out of its own O buffer while the softmax works on
// Every wait is bounded, by some 2 s; a wait that gives up sets TS_STATUS_TIMEOUT,
// the others follow by their own limits or the group's vote (a warp waits in vain
// three times at most), and TMEM is freed.
//
// Bounds, measured. A tile of 128 keys (33 KB at d = 128) has to pass an SM in
// 0.74 us at the measured copy peak of 6.8 TB/s, and does with 16 rows a unit
// (64 requests x 56 heads x 1040 keys: 152 us, 98% of the peak). With more rows
// the softmax warps' latency bounds it: 32 rows 183 us (85%), 47 rows 205 us
// (79%; 94% over 8192 keys), where a unit of 9 tiles costs some 2 us beside its
// tiles (first maxima, masked tile, sums). 64 rows take 0.8 us a tile (4 x 64
// heads x 16512 keys x 128 nodes: 395 us, 696 TFLOP/s of attention arithmetic). What carried it
// there: two tiles of scores and two of probabilities in flight; one wait a tile
// for both; no branch and few instructions in the common tile (its loop has to
// stay in the instruction cache: a version of twice the code took 1.4 times as
// long); units switched by other warps than the softmax's. A call of few tiles
// is bound by its chain: 5 us until the plan is made and the first scores are
// there, 3 us for the output and the join of cut items (8 requests of one token
// over 2048 keys: 14.7 us, 5.1 us at the copy peak).
#include <cuda.h>
#include <math.h>

#include "attn_common.cuh"
#include "kv8.cuh"
#include "kv8_wait.cuh"

namespace ts {
namespace {

// ---------------------------------------------------------------- PTX ---
__device__ __forceinline__ uint64_t smem_desc8(uint32_t addr, uint32_t lbo, uint32_t sbo, uint64_t layout) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)((lbo >> 4) & 0x3FFFu) << 16 |
           (uint64_t)((sbo >> 4) & 0x3FFFu) << 32 | (uint64_t)1 << 46 | layout << 61;
}
constexpr uint64_t kSwz128 = 2, kSwz64 = 4;

// kind::f8f6f4 instruction descriptor: fp32 accumulate, A e4m3, B e4m3 or e5m2.
constexpr uint32_t idesc_f8(int M, int N, bool b_e5m2, bool a_mn, bool b_mn) {
    return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
        ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}

__device__ __forceinline__ void tc_ld8(uint32_t taddr, float *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tc_ld4(uint32_t taddr, float *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(taddr));
}
__device__ __forceinline__ void tc_st4(uint32_t taddr, const float *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "f"(v[0]), "f"(v[1]),
                 "f"(v[2]), "f"(v[3])
                 : "memory");
}

template <int N>
__device__ __forceinline__ void tc_ldn(uint32_t taddr, float (&v)[N]) {
    if constexpr (N == 16) tc_ld16(taddr, v);
    else tc_ld8(taddr, v);
}

// Maximum over the warp, NaN left out.
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// log2 of a normal number.
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Barrier of `threads` threads that also tells whether any of them votes.
__device__ __forceinline__ bool bar_any(int id, int threads, bool vote) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"((uint32_t)vote), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// 4-byte asynchronous copy to shared memory; zeros where !valid.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
// One arrival of this thread once its copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Shared memory by its 32-bit address.
__device__ __forceinline__ float4 lds4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float lds1(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ int ldsi(uint32_t a) {
    int v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void sts1(uint32_t a, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void stsi(uint32_t a, int v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts4u(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void sts2u(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t half2_to_fp8x2(uint32_t h) {
    __half2_raw r;
    r.x = (unsigned short)h;
    r.y = (unsigned short)(h >> 16);
    return __nv_cvt_halfraw2_to_fp8x2(r, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t fp8x2_to_half2(uint32_t c) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3);
    return (uint32_t)r.x | (uint32_t)r.y << 16;
}
// ------------------------------------------------------------ arguments ---
struct Attn8Args {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    const float *k_scale, *v_scale;
    const int32_t *prefix_len;
    ts_tree t;
    int Hq, H, G, rows;   // rows: L_max of the cache
    float scale_log2;
    PagedArgs pg;
    uint32_t *status;
    unsigned *queue;      // [0] next unit, [1] CTAs finished
    unsigned *joins;      // [slots] parts done, by the item's first slot
    float2 *part_ml;      // [slots][RP] (maximum, sum)
    float *part_o;        // [slots][RP][D]
    int slots;
};

constexpr int kTileKeys = 128;
constexpr int kReqCache = 128;     // requests planned in shared memory
constexpr int kMaxCuts = 32;       // parts of one item (a lane each when they are joined)
constexpr int kMinCut = 3;         // tiles of a part at least
constexpr int kSlotsPerSm = 12;    // parts of cut items there is room for
constexpr float kUnitCost = 5.f, kJoinCost = 6.f;   // of a unit beside its tiles, and of joining parts, in tiles
constexpr int kRing = 4;           // published units
constexpr int kClaimAhead = 10;    // tiles

template <int D_, int RP_>
struct Cfg8 {
    static constexpr int D = D_, RP = RP_, CG = RP <= 32 ? 8 : 16, GROUPS = RP / CG;   // columns of a softmax group
    static constexpr int SM_WARPS = 4 * GROUPS, THREADS = 32 * (4 + SM_WARPS + 4);
    // Registers a thread where SPLIT: LAUNCH x THREADS at launch, handed from the eight other warps to the softmax's where 65536 /
    // THREADS does not do for those. RP = 48: 640 x 96 = 61440 >= 256 x 80 + 384 x 104 = 60416; 64: 768 x 80 = 61440 =
    // 256 x 64 + 512 x 88. (With 56 and 48 for the others short units, whose output counts, take up to a quarter longer,
    // long ones 1% less.)
    static constexpr bool SPLIT = RP >= 48;
    static constexpr int LAUNCH_REGS = RP == 64 ? 80 : 96, SM_REGS = RP == 64 ? 88 : 104, OTHER_REGS = RP == 64 ? 64 : 80;
    static_assert(!SPLIT || 32 * SM_WARPS * SM_REGS + 256 * OTHER_REGS <= THREADS * LAUNCH_REGS, "a split of the launch's registers");
    static constexpr int OP_BYTES = kTileKeys * D;             // codes of one operand tile
    static constexpr int STAGE_BYTES = 2 * OP_BYTES;
    static constexpr int P_ATOMS = (3 * RP + 63) / 64, P_ATOM = kTileKeys * 64, P_BYTES = P_ATOMS * P_ATOM;
    static constexpr int Q_BYTES = 2 * RP * D;
    static constexpr int SIDE = 3 * kTileKeys * 4;             // a stage's key scales, value scales, subtree ends
    // fixed part, behind the stages
    static constexpr int FIX_P = 0, FIX_Q = FIX_P + 2 * P_BYTES, FIX_MX = FIX_Q + 2 * Q_BYTES;
    static constexpr int FIX_F2 = FIX_MX + 4 * RP * 4;         // column maxima [groups][4 warps][CG]; roots of O's factors [64]
    static constexpr int FIX_M = FIX_F2 + 64 * 4;              // kBase - maximum [64]
    static constexpr int FIX_SUM = FIX_M + 64 * 4, SUM_BYTES = 5 * 64 * 4;   // by unit parity: column sums [4 warps][64], maxima [64]
    static constexpr int FIX_QS = FIX_SUM + 2 * SUM_BYTES;     // query scales [kRing][64], output rows [kRing][64]
    static constexpr int FIX_QROW = FIX_QS + kRing * 64 * 4;
    static constexpr int FIX_REQ = FIX_QROW + kRing * 64 * 4;  // requests: n, P, tiles, parts
    static constexpr int FIX_KEY = FIX_REQ + kReqCache * 16;   // tiles of a part
    static constexpr int FIX_ORDER = FIX_KEY + kReqCache * 4;  // by rank: request, first unit, first slot
    static constexpr int FIX_UNIT = FIX_ORDER + kReqCache * 4, FIX_SLOT = FIX_UNIT + kReqCache * 4;
    static constexpr int FIX_INFO = FIX_SLOT + kReqCache * 4;  // units [kRing][12]
    static constexpr int FIX_MISC = FIX_INFO + kRing * 12 * 4; // 0 TMEM base, 1 timeout, 3 last
    static constexpr int FIX_BAR = FIX_MISC + 64;
    static constexpr int FIX_END = FIX_BAR + 64 * 8;
    static constexpr int off_fix(int stages) { return (stages * (STAGE_BYTES + SIDE) + 1023) / 1024 * 1024; }
    static constexpr int fit() {
        int n = 8;
        while (off_fix(n) + FIX_END + 1024 > 232448) --n;
        return n;
    }
    static constexpr int STAGES = fit();
    static constexpr int OFF_SIDE = STAGES * STAGE_BYTES, OFF_FIX = off_fix(STAGES), SMEM = OFF_FIX + FIX_END + 1024;
    static constexpr uint32_t S_COL = 0, O_COL = 2 * RP;       // two score buffers of RP columns, two O of 3 RP
    static constexpr uint32_t TMEM_COLS = 8 * RP <= 128 ? 128 : 8 * RP <= 256 ? 256 : 512;
    static_assert(STAGES >= 4 && SMEM <= 232448 && STAGE_BYTES % 1024 == 0 && FIX_Q % 1024 == 0 && Q_BYTES % 1024 == 0,
                  "shared memory and the alignment of swizzled tiles");
};

struct Unit8 {
    int b, h, row0, n, P, j0, j1, parts, part, slot;   // tiles [j0, j1); slot: of the item's first part
};

// Sums of N columns over the warp: column lane / (32 / N) ends in v[0].
template <int N, int W = 16>
__device__ __forceinline__ void reduce_scatter(float *v, int lane) {
    if constexpr (N > 1) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float keep = lane & W ? v[i + N / 2] : v[i], send = lane & W ? v[i] : v[i + N / 2];
            v[i] = keep + __shfl_xor_sync(~0u, send, W);
        }
    } else {
        v[0] += __shfl_xor_sync(~0u, v[0], W);
    }
    if constexpr (W > 1) reduce_scatter<(N > 1 ? N / 2 : 1), W / 2>(v, lane);
}

// The parts of a cut item into its output rows, by four warps with RP / 4 columns each.
template <int D, int RP>
__device__ __forceinline__ void join_parts(const float2 *part_ml, const float *part_o, int parts, uint32_t rows,
                                           __nv_bfloat16 *out) {
    const int lane = threadIdx.x & 31;
    __threadfence();
    if constexpr (RP == 16) {
        // a column at a time, lane = part for its weights, then dims: the least code, which counts for a loop that runs
        // four times, cold (one request of one token over 2048 keys: 11.2 us against 12.6)
        constexpr int EPL = D / 32;
#pragma unroll 1
        for (int c = (threadIdx.x >> 5) & 3; c < RP; c += 4) {
            const int row = ldsi(rows + c * 4);
            if (row < 0) continue;
            float2 ml = make_float2(-INFINITY, 0.f);
            if (lane < parts) ml = __ldcg(part_ml + (size_t)lane * RP + c);
            const float mx = warp_max(ml.x);
            // a part of small values may have large sums: its weight, which alone may be below fp32's range, in two steps
            const float root = lane < parts ? ex2(0.5f * (ml.x - mx)) : 0.f, wt = root * root;
            float ls = root * ml.y * root;
#pragma unroll
            for (int o = 16; o; o >>= 1) ls += __shfl_xor_sync(~0u, ls, o);
            float acc[EPL] = {};
            const float *po = part_o + (size_t)c * D + lane * EPL;
#pragma unroll 4
            for (int s = 0; s < parts; ++s) {
                const float ws = __shfl_sync(~0u, wt, s);
                float v[EPL];
                if constexpr (EPL == 4) {
                    const float4 f = __ldcg((const float4 *)(po + (size_t)s * RP * D));
                    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
                } else {
                    const float2 f = __ldcg((const float2 *)(po + (size_t)s * RP * D));
                    v[0] = f.x; v[1] = f.y;
                }
#pragma unroll
                for (int e = 0; e < EPL; ++e) acc[e] = fmaf(ws, v[e], acc[e]);
            }
            const float inv = 1.f / ls;
#pragma unroll
            for (int e = 0; e < EPL; e += 2)
                *(__nv_bfloat162 *)(out + (size_t)row * D + lane * EPL + e) = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
        }
    } else {
        // every column's maximum and sum first (lane = column, half of the parts), then two columns at a time, whose
        // loads do not wait for one another (4 x 128 nodes, 64 heads, 16384 keys: 393 us against 403)
        constexpr int COLS = RP / 4, EPL = D / 16, AHEAD = RP == 64 ? 1 : 4;   // more code costs more than it hides
        const int c0 = ((threadIdx.x >> 5) & 3) * COLS;
        const int mine = c0 + min(lane & 15, COLS - 1);
        float mx = -1e38f, sum = 0.f;
#pragma unroll 4
        for (int s = lane >> 4; s < parts; s += 2) {
            const float2 ml = __ldcg(part_ml + (size_t)s * RP + mine);
            const float top = fmaxf(mx, ml.x), f = ex2(0.5f * (mx - top)), g = ex2(0.5f * (ml.x - top));   // roots: as above
            sum = f * sum * f + g * ml.y * g;
            mx = top;
        }
        const float mo = __shfl_xor_sync(~0u, mx, 16), so = __shfl_xor_sync(~0u, sum, 16), top = fmaxf(mx, mo);
        const float fm = ex2(0.5f * (mx - top)), fo = ex2(0.5f * (mo - top)), a = fm * sum * fm, b = fo * so * fo;
        const float inv = 1.f / (a + b);
        mx = top;
#pragma unroll 1
        for (int i = lane >> 4; i < COLS; i += 2) {
            const float m = __shfl_sync(~0u, mx, i), f = __shfl_sync(~0u, inv, i);
            const int c = c0 + i, row = ldsi(rows + c * 4);
            float acc[EPL] = {};
            const float2 *pm = part_ml + c;
            const float *po = part_o + (size_t)c * D + (lane & 15) * EPL;
#pragma unroll AHEAD
            for (int s = 0; s < parts; ++s, pm += RP, po += (size_t)RP * D) {
                const float w = ex2(__ldcg(&pm->x) - m);
#pragma unroll
                for (int e = 0; e < EPL; e += 4) {
                    const float4 v = __ldcg((const float4 *)(po + e));
                    acc[e] = fmaf(w, v.x, acc[e]);
                    acc[e + 1] = fmaf(w, v.y, acc[e + 1]);
                    acc[e + 2] = fmaf(w, v.z, acc[e + 2]);
                    acc[e + 3] = fmaf(w, v.w, acc[e + 3]);
                }
            }
            if (row >= 0) {
                __nv_bfloat162 v[EPL / 2];
#pragma unroll
                for (int e = 0; e < EPL / 2; ++e) v[e] = __floats2bfloat162_rn(acc[2 * e] * f, acc[2 * e + 1] * f);
                __nv_bfloat16 *to = out + (size_t)row * D + (lane & 15) * EPL;
                if constexpr (EPL == 8) *(uint4 *)to = *(const uint4 *)v;
                else *(uint2 *)to = *(const uint2 *)v;
            }
        }
    }
}

template <bool MORE, int N>
__device__ __forceinline__ void take_registers() {
    if constexpr (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D, int RP>
__global__ void __launch_bounds__(Cfg8<D, RP>::THREADS, 1)
    k_attn_kv8(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, Attn8Args a) {
    using C = Cfg8<D, RP>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *sm = (unsigned char *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    unsigned char *fix = sm + C::OFF_FIX;
    const uint32_t sm_base = smem_u32(sm), fix_base = sm_base + C::OFF_FIX;
    volatile int *misc = (volatile int *)(fix + C::FIX_MISC);
    int4 *req_s = (int4 *)(fix + C::FIX_REQ);
    int *key_s = (int *)(fix + C::FIX_KEY), *order_s = (int *)(fix + C::FIX_ORDER);
    int *unit_s = (int *)(fix + C::FIX_UNIT), *slot_s = (int *)(fix + C::FIX_SLOT);
    float *cost_s = (float *)slot_s;   // until the way of cutting is picked

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int B = a.t.B, n_max = a.t.n_max;

    const uint32_t full = fix_base + C::FIX_BAR, empty = full + 8 * C::STAGES, sfull = empty + 8 * C::STAGES;
    const uint32_t pvdone = sfull + 16, pfull = pvdone + 16, qraw = pfull + 16, qready = qraw + 16, qfree = qready + 16;
    const uint32_t fin = qfree + 16, sumfull = fin + 16, odone = sumfull + 16, ofree = odone + 16;
    const uint32_t iready = ofree + 16, ifree = iready + 8 * kRing, claimgo = ifree + 8 * kRing;

    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32((void *)misc)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
#pragma unroll 1
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(full + 8 * s, 1 + 32);   // the TMA's bytes, and the producer's lanes' copies
            mbar_init(empty + 8 * s, 1);
        }
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
            // the scores, the issuer's sight of the stage (scales by cp.async), and the product two tiles before, which
            // has read the probabilities that this tile's overwrite (with a wait of its own for that, the long-context
            // case took 452 us instead of 424)
            mbar_init(sfull + 8 * x, 3);
            mbar_arrive(sfull + 8 * x);   // there is no such product yet
            mbar_init(pvdone + 8 * x, 1);
            mbar_init(pfull + 8 * x, C::SM_WARPS);
            mbar_init(qraw + 8 * x, 1 + 32);
            mbar_init(qready + 8 * x, 4);
            mbar_init(sumfull + 8 * x, C::SM_WARPS);
            mbar_init(odone + 8 * x, 1);
            mbar_init(ofree + 8 * x, 4);
            mbar_init(qfree + 8 * x, 1);
            mbar_init(fin + 8 * x, 1);
        }
#pragma unroll 1
        for (int r = 0; r < kRing; ++r) {
            mbar_init(iready + 8 * r, 1);
            mbar_init(ifree + 8 * r, 3 + C::SM_WARPS + 4);
        }
        mbar_init(claimgo, 1);
        misc[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }

    if (tid < 2) {
        const CUtensorMap *map = tid ? &map_v : &map_k;
        asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
    }
    pdl_wait();   // nothing above touches global memory
    pdl_trigger();

    // ---- the plan, the same in every CTA: how many tiles a part has, and each
    // request's first unit and first slot of the workspace
    const bool planned = B <= kReqCache;
    auto blocks_of = [&](int n) { return (n * a.G + RP - 1) / RP; };
    auto tiles_of = [&](int n, int P) -> int {   // 0 for a request that is empty or does not fit
        return n > 0 && n <= n_max && P >= 0 && P <= a.rows - n ? (P + n + kTileKeys - 1) / kTileKeys : 0;
    };
    // a part's tiles for way i of cutting, and an item's parts by its reciprocal (taken a little low, so that whole
    // quotients stay so: these are approximate divisions, the same in every CTA)
    auto part_tiles = [](int longest, int i) {
        return fmaxf((float)kMinCut, ceilf(__fdividef((float)longest, (float)(i + 1)) * 0.999999f));
    };
    auto parts_of = [](int tiles, float rate) { return fminf(ceilf(tiles * rate), (float)kMaxCuts); };
    auto rate_of = [](float per) { return __fdividef(0.999999f, per); };
    int ticket = 0;   // the CTA's first place in the queue
    if (warp == 3 && lane == 0) ticket = (int)atomicAdd(a.queue, 1u);
#pragma unroll 1
    for (int b = tid; b < B; b += C::THREADS) {
        const int n = a.t.n_nodes[b], P = a.prefix_len[b], tl = tiles_of(n, P);
        if (planned) req_s[b] = make_int4(n, P, tl, 1);
        if (blockIdx.x == 0 && n > 0 && !tl) flag(a.status, TS_STATUS_INDEX);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)misc[0];
    int longest = 0, same = 1;   // same: tiles and row blocks of every request
    if (planned) {
        const int4 rq0 = req_s[0];
#pragma unroll 1
        for (int b = lane; b < B; b += 32) {
            const int4 rq = req_s[b];
            longest = max(longest, rq.z);
            same &= rq.z == rq0.z && blocks_of(rq.x) == blocks_of(rq0.x);
        }
        longest = __reduce_max_sync(~0u, longest);
        same = __all_sync(~0u, same);
    }
    const bool cuts = longest > kMinCut;   // no item can be cut otherwise
    if (cuts) {
        // How far to cut: parts of at most 1 / (i + 1) of the longest item, half a warp for each of 32 ways (lane =
        // request). Items of one length take as many rounds over the SMs as they have units; others, handed out
        // longest first, about their sum over the SMs and half a longest unit. Cut items have to fit the slots.
        static_assert(C::THREADS >= 16 * 32, "half a warp a way");
        const int i = tid >> 4;
        if (warp < 16) {
            const float per = part_tiles(longest, i), rate = rate_of(per);
            float work = 0.f, units = 0.f, cut = 0.f;   // tiles, units, units of cut items
#pragma unroll 1
            for (int b = lane & 15; b < B; b += 16) {
                const int4 rq = req_s[b];
                const float items = (float)(a.H * blocks_of(rq.x)), parts = parts_of(rq.z, rate);
                work += items * rq.z;
                units += items * parts;
                cut += parts > 1.f ? items * parts : 0.f;
            }
#pragma unroll
            for (int o = 8; o; o >>= 1) {
                work += __shfl_xor_sync(~0u, work, o);
                units += __shfl_xor_sync(~0u, units, o);
                cut += __shfl_xor_sync(~0u, cut, o);
            }
            const float all = work + units * kUnitCost, sms = (float)gridDim.x;
            const float spread = same ? ceilf(__fdividef(units, sms) * 0.999999f) * __fdividef(all, fmaxf(units, 1.f))
                                      : __fdividef(all, sms) + 0.5f * per;
            float cost = fmaxf(per + kUnitCost, spread) + (cut > 0.f ? kJoinCost : 0.f);
            if (i > 0 && cut > (float)a.slots) cost = 3e38f;
            if ((lane & 15) == 0) cost_s[i] = cost;
        }
        __syncthreads();
    }

    auto read_unit = [&](int r) -> Unit8 {
        const uint32_t i = fix_base + C::FIX_INFO + r * 48;
        const float4 v = lds4(i), w = lds4(i + 16), x = lds4(i + 32);
        return Unit8{__float_as_int(v.x), __float_as_int(v.y), __float_as_int(v.z), __float_as_int(v.w), __float_as_int(w.x),
                     __float_as_int(w.y), __float_as_int(w.z), __float_as_int(w.w), __float_as_int(x.x), __float_as_int(x.y)};
    };

    constexpr uint64_t swz = D == 128 ? kSwz128 : kSwz64;
    if (warp < 4) {
        if constexpr (C::SPLIT) take_registers<false, C::OTHER_REGS>();
        if (warp == 0) {   // ------------------------------------------------ producer
            int g = 0;
            bool ok = true;
#pragma unroll 1
            for (int k = 0; ok; ++k) {
                const int r = k % kRing;
                if (!wait_warp(iready + 8 * r, (uint32_t)(k / kRing) & 1u)) {
                    ok = false;
                    break;
                }
                const Unit8 u = read_unit(r);
                __syncwarp();
                if (lane == 0) mbar_arrive(ifree + 8 * r);
                if (u.b < 0) break;
                const int claim = max(u.j1 - kClaimAhead, u.j0);
                const int L = u.P + u.n;
                const int strip = (u.b * a.H + u.h) * a.rows;   // dense: the cache row of key 0
#pragma unroll 1
                for (int j = u.j0; j < u.j1; ++j, ++g) {
                    if (j == claim && lane == 0) mbar_arrive(claimgo);
                    const int st = g % C::STAGES, key0 = j * kTileKeys;
                    const bool two = key0 + 64 < L;
                    int row0 = strip + key0, row1 = row0 + 64;
                    bool has0 = true, has1 = true;
                    if (a.pg.bt) {   // a page's 64 rows of this head; zeros (a row far outside) for a page that is none
                        const int32_t *bt = a.pg.bt + (size_t)u.b * a.pg.max_pages + key0 / TS_PAGE_KEYS;
                        const int p0 = __ldg(bt), p1 = two ? __ldg(bt + 1) : 0;
                        has0 = p0 >= 0 && p0 < a.pg.num_pages;
                        has1 = p1 >= 0 && p1 < a.pg.num_pages;
                        if (lane == 0 && !(has0 && has1)) flag(a.status, TS_STATUS_INDEX);
                        row0 = has0 ? (p0 * a.H + u.h) * TS_PAGE_KEYS : 0x7fffff00;
                        row1 = has1 ? (p1 * a.H + u.h) * TS_PAGE_KEYS : 0x7fffff00;
                    }
                    if (g >= C::STAGES && !wait_warp(empty + 8 * st, (uint32_t)(g / C::STAGES - 1) & 1u)) {
                        ok = false;
                        break;
                    }
                    const uint32_t kd = sm_base + st * C::STAGE_BYTES, vd = kd + C::OP_BYTES, fb = full + 8 * st;
                    if (lane == 0) {
                        if (a.pg.bt) {
                            mbar_expect_tx(fb, (two ? 4 : 2) * 64 * D);
                            tma_load_2d(kd, &map_k, 0, row0, fb);
                            tma_load_2d(vd, &map_v, 0, row0, fb);
                            if (two) {
                                tma_load_2d(kd + 64 * D, &map_k, 0, row1, fb);
                                tma_load_2d(vd + 64 * D, &map_v, 0, row1, fb);
                            }
                        } else {
                            mbar_expect_tx(fb, C::STAGE_BYTES);
                            tma_load_2d(kd, &map_k, 0, row0, fb);
                            tma_load_2d(vd, &map_v, 0, row0, fb);
                        }
                    }
                    const uint32_t side = sm_base + C::OFF_SIDE + st * C::SIDE + lane * 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool in = key0 + i * 32 + lane < L && (i < 2 ? has0 : has1);
                        const int row = in ? (i < 2 ? row0 : row1) + (i & 1) * 32 + lane : 0;
                        cp_async4(side + i * 128, a.k_scale + row, in);
                        cp_async4(side + 512 + i * 128, a.v_scale + row, in);
                    }
                    if (key0 + kTileKeys > u.P) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int node = key0 + i * 32 + lane - u.P;
                            const bool in = node >= 0 && node < u.n;
                            cp_async4(side + 1024 + i * 128, a.t.sub_end + (in ? (size_t)u.b * n_max + node : 0), in);
                        }
                    }
                    cp_async_arrive(fb);
                }
            }
            if (!ok) {   // leave no copy in flight; one that does not land in a wait's time is the last that is waited for
                if (lane == 0) misc[1] = 1;
#pragma unroll 1
                for (int i = g > C::STAGES ? g - C::STAGES : 0; i < g; ++i)
                    if (!wait_warp(full + 8 * (i % C::STAGES), (uint32_t)(i / C::STAGES) & 1u)) break;
            }
        } else if (warp == 1) {   // ----------------------------------------- MMA issuer
            if (lane == 0) {
                constexpr uint32_t idesc_s = idesc_f8(128, RP, false, false, false);
                bool ok = true;
                int g = 0;
                for (int k = 0; ok; ++k) {
                    const int r = k % kRing;
                    if (!wait1(iready + 8 * r, (uint32_t)(k / kRing) & 1u)) { ok = false; break; }
                    const Unit8 u = read_unit(r);
                    mbar_arrive(ifree + 8 * r);
                    if (u.b < 0) break;
                    if (!wait1(qready + 8 * (k & 1), (uint32_t)(k >> 1) & 1u)) { ok = false; break; }
#pragma unroll 1
                    for (int j = u.j0; j < u.j1; ++j, ++g) {
                        const int st = g % C::STAGES, x = g & 1;
                        // once the probabilities of tile g - 2 are there S(g - 2) has been read; their product need not be done
                        if ((g >= 2 && !wait1(pfull + 8 * x, (uint32_t)((g - 2) >> 1) & 1u)) ||
                            !wait1(full + 8 * st, (uint32_t)(g / C::STAGES) & 1u)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t kb = sm_base + st * C::STAGE_BYTES, qd = fix_base + C::FIX_Q + (k & 1) * C::Q_BYTES;
#pragma unroll
                        for (int kk = 0; kk < 2 * (D / 32); ++kk)   // with the rows' upper, then their lower parts
                            tc_mma_f8(tmem + C::S_COL + x * RP, smem_desc8(kb + kk % (D / 32) * 32, 16, 8 * D, swz),
                                      smem_desc8(qd + kk / (D / 32) * RP * D + kk % (D / 32) * 32, 16, 8 * D, swz), idesc_s, kk > 0);
                        tc_commit(sfull + 8 * x);
                        mbar_arrive(sfull + 8 * x);
                    }
                    if (ok) tc_commit(qfree + 8 * (k & 1));   // the unit's query rows may be overwritten
                }
                if (!ok) misc[1] = 1;
                tc_commit(fin);
                if (!wait1(fin, 0)) misc[1] = 1;
            }
            __syncwarp();
        } else if (warp == 2) {   // ----------------------------------------- O += P V
            // a thread of its own: a product waits for its tile's probabilities only, never for the next tile's load
            if (lane == 0) {
                constexpr uint32_t idesc_o = idesc_f8(128, 3 * RP, true, true, true);
                bool ok = true;
                int g = 0;
                for (int k = 0; ok; ++k) {
                    const int r = k % kRing;
                    if (!wait1(iready + 8 * r, (uint32_t)(k / kRing) & 1u)) { ok = false; break; }
                    const Unit8 u = read_unit(r);
                    mbar_arrive(ifree + 8 * r);
                    if (u.b < 0) break;
                    if (k >= 2 && !wait1(ofree + 8 * (k & 1), (uint32_t)(k / 2 - 1) & 1u)) { ok = false; break; }
#pragma unroll 1
                    for (int j = u.j0; j < u.j1; ++j, ++g) {
                        const int st = g % C::STAGES, x = g & 1;
                        if (!wait1(full + 8 * st, (uint32_t)(g / C::STAGES) & 1u) ||
                            !wait1(pfull + 8 * x, (uint32_t)(g >> 1) & 1u)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t vb = sm_base + st * C::STAGE_BYTES + C::OP_BYTES, pd = fix_base + C::FIX_P + x * C::P_BYTES;
                        // a unit's first product starts its O afresh; the buffer's last one has been read out.
                        // V^T: dims contiguous; d = 64 repeats its 64 rows (stride 0) to the MMA's 128
#pragma unroll
                        for (int kk = 0; kk < kTileKeys / 32; ++kk)
                            tc_mma_f8(tmem + C::O_COL + (k & 1) * 3 * RP, smem_desc8(vb + kk * 32 * D, 0, 8 * D, swz),
                                      smem_desc8(pd + kk * 32 * 64, C::P_ATOM, 512, kSwz64), idesc_o, j > u.j0 || kk > 0);
                        tc_commit(empty + 8 * st);
                        tc_commit(pvdone + 8 * x);
                        tc_commit(sfull + 8 * x);
                    }
                    if (ok) tc_commit(odone + 8 * (k & 1));
                }
                if (!ok) misc[1] = 1;
                tc_commit(fin + 8);
                if (!wait1(fin + 8, 0)) misc[1] = 1;
            }
            __syncwarp();
        } else if (warp == 3) {   // ----------------------------------------- queue and query rows
            // ---- the rest of the plan
            int units = 0;
            if (planned) {
                int pick = 0;
                if (cuts) {
                    // the way of the least cost (costs are positive: their bits order as they do), the least cutting of
                    // equal ones
                    const uint32_t cost = __float_as_uint(cost_s[lane]), least = __reduce_min_sync(~0u, cost);
                    pick = __ffs(__ballot_sync(~0u, cost == least)) - 1;
                }
                const float rate = rate_of(part_tiles(longest, pick));
                if (same) {
                    const int4 rq = req_s[0];
                    const int parts = max(1, (int)parts_of(rq.z, rate)), u = rq.z ? a.H * blocks_of(rq.x) * parts : 0;
                    __syncwarp();
#pragma unroll 1
                    for (int b = lane; b < B; b += 32) {
                        req_s[b].w = parts;
                        order_s[b] = b;
                        unit_s[b] = b * u;
                        slot_s[b] = parts > 1 ? b * u : 0;
                    }
                    units = B * u;
                } else {
#pragma unroll 1
                    for (int b = lane; b < B; b += 32) {
                        const int tl = req_s[b].z, parts = max(1, (int)parts_of(tl, rate));
                        req_s[b].w = parts;
                        key_s[b] = parts > 1 ? (tl + parts - 1) / parts : tl;
                    }
                    __syncwarp();
                    // requests by the length of their parts, longest first
#pragma unroll 1
                    for (int b = lane; b < B; b += 32) {
                        int rank = 0;
                        const int mine = key_s[b];
#pragma unroll 4
                        for (int o = 0; o < B; ++o) {
                            const int ko = key_s[o];
                            rank += ko > mine || (ko == mine && o < b);
                        }
                        order_s[rank] = b;
                    }
                    __syncwarp();
                    // exclusive sums of units and of slots, in that order
                    int ns = 0;
#pragma unroll 1
                    for (int r0 = 0; r0 < B; r0 += 32) {
                        int u = 0, c = 0;
                        if (r0 + lane < B) {
                            const int4 rq = req_s[order_s[r0 + lane]];
                            if (rq.z) u = a.H * blocks_of(rq.x) * rq.w;
                            if (rq.w > 1) c = u;
                        }
                        int cu = u, cc = c;
#pragma unroll 1
                        for (int o = 1; o < 32; o <<= 1) {
                            const int tu = __shfl_up_sync(~0u, cu, o), tc = __shfl_up_sync(~0u, cc, o);
                            if (lane >= o) {
                                cu += tu;
                                cc += tc;
                            }
                        }
                        if (r0 + lane < B) {
                            unit_s[r0 + lane] = units + cu - u;
                            slot_s[r0 + lane] = ns + cc - c;
                        }
                        units += __shfl_sync(~0u, cu, 31);
                        ns += __shfl_sync(~0u, cc, 31);
                    }
                }
                __syncwarp();
            } else {
                units = B * a.H * ((n_max * a.G + RP - 1) / RP);
            }
            // unit q of the queue; false for one that is empty (requests beyond the planned ones)
            auto decode = [&](int q, Unit8 &u) -> bool {
                int first, tl, blocks;
                u.slot = 0;
                u.parts = 1;
                if (planned) {
                    int lo = 0, hi = B - 1;   // the last request whose first unit is at most q
#pragma unroll 1
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (unit_s[mid] <= q) lo = mid;
                        else hi = mid - 1;
                    }
                    u.b = order_s[lo];
                    first = unit_s[lo];
                    u.slot = slot_s[lo];
                    const int4 rq = req_s[u.b];
                    u.n = rq.x;
                    u.P = rq.y;
                    tl = rq.z;
                    u.parts = rq.w;
                    blocks = blocks_of(u.n);
                } else {
                    blocks = (n_max * a.G + RP - 1) / RP;
                    u.b = q / (a.H * blocks);
                    first = u.b * a.H * blocks;
                    u.n = a.t.n_nodes[u.b];
                    u.P = a.prefix_len[u.b];
                    tl = tiles_of(u.n, u.P);
                }
                // row blocks of the same keys follow one another: the second finds them in L2
                const int rest = q - first, item = blocks > 1 ? rest / blocks : rest, blk = rest - item * blocks;
                u.part = u.parts > 1 ? item / a.H : 0;
                u.h = item - u.part * a.H;
                u.row0 = blk * RP;
                if (!tl || blk >= blocks_of(u.n)) return false;
                u.j0 = 0;
                u.j1 = tl;
                if (u.parts > 1) {   // parts differ by a tile at most
                    const int len = tl / u.parts, rem = tl - len * u.parts;
                    u.j0 = u.part * len + min(u.part, rem);
                    u.j1 = u.j0 + len + (u.part < rem);
                    u.slot += (u.h * blocks + blk) * u.parts;
                }
                return true;
            };
            // A raw row of 2 * d bytes and its two parts of d bytes take the same room: each half of the row is copied
            // to where a part will be; the output warps turn rows into parts in place.
            bool ok = true;
            for (int k = 0;; ++k) {
                // the next unit is taken kClaimAhead tiles before the last load of the one before, late enough that CTAs
                // share the last units evenly, early enough that its query rows are staged in time
                int q = ticket;
                if (k > 0) {
                    if (!wait_warp(claimgo, (uint32_t)(k - 1) & 1u)) { ok = false; break; }
                    if (lane == 0) q = (int)atomicAdd(a.queue, 1u);
                }
                q = __shfl_sync(~0u, q, 0);
                Unit8 u = {};
                while (q < units && !decode(q, u)) {
                    if (lane == 0) q = (int)atomicAdd(a.queue, 1u);
                    q = __shfl_sync(~0u, q, 0);
                }
                const int r = k % kRing;
                if (k >= kRing && !wait_warp(ifree + 8 * r, (uint32_t)(k / kRing - 1) & 1u)) { ok = false; break; }
                if (lane == 0) {
                    const uint32_t i = fix_base + C::FIX_INFO + r * 48;
                    const int v[10] = {q < units ? u.b : -1, u.h, u.row0, u.n, u.P, u.j0, u.j1, u.parts, u.part, u.slot};
#pragma unroll
                    for (int e = 0; e < 10; ++e) stsi(i + 4 * e, v[e]);
                    mbar_arrive(iready + 8 * r);
                }
                if (q >= units) break;
                // lane i looks up the places of rows i and 32 + i of the block in q and out
                int place[2] = {-1, -1};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = h * 32 + lane;
                    if (c < RP) {
                        const int rho = u.row0 + c, i = rho / a.G;
                        if (i < u.n) {
                            const int v = a.t.perm[(size_t)u.b * n_max + i];
                            if (v >= 0 && v < n_max) place[h] = v * a.Hq + u.h * a.G + (rho - i * a.G);
                        }
                        stsi(fix_base + C::FIX_QROW + (r * 64 + c) * 4, place[h]);
                    }
                }
                if (k >= 2 && !wait_warp(qfree + 8 * (k & 1), (uint32_t)(k / 2 - 1) & 1u)) { ok = false; break; }
                const uint32_t qd = fix_base + C::FIX_Q + (k & 1) * C::Q_BYTES;
                const __nv_bfloat16 *qb = a.q + (size_t)u.b * n_max * a.Hq * D;
                constexpr int VPR = D / 8;   // 16-byte pieces of a raw row
#pragma unroll 4
                for (int i = lane; i < RP * VPR; i += 32) {
                    const int c = i / VPR, v = i % VPR;
                    const int lo = __shfl_sync(~0u, place[0], c & 31), hi = __shfl_sync(~0u, place[1], c & 31);
                    const int pl = c < 32 ? lo : hi;
                    cp_async16(qd + ((v >= VPR / 2 ? RP : 0) + c) * D + (v % (VPR / 2)) * 16,
                               qb + (size_t)(pl < 0 ? 0 : pl) * D + v * 8, pl >= 0);
                }
                cp_async_arrive(qraw + 8 * (k & 1));
                __syncwarp();
                if (lane == 0) mbar_arrive(qraw + 8 * (k & 1));   // hands on the rows' places
            }
            if (!ok && lane == 0) misc[1] = 1;
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else if (warp < 4 + C::SM_WARPS) {   // ---------------------------- softmax
        if constexpr (C::SPLIT) take_registers<true, C::SM_REGS>();
        constexpr int CG = C::CG;
        // w is 2^kBase at the reference, which is raised once a key's y + log2(vs) passes it by 2^kOver: fp16 (and e5m2) hold
        // both ends, and a weight of 2^-23 of the reference's still has a bit
        constexpr float kBase = 7.f, kOver = 8.f;
        const int grp = (warp - 4) >> 2, quarter = warp & 3, cb = grp * CG;
        const int bar = 1 + grp, gt = quarter * 32 + lane;   // thread of the group
        const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
        const int kslot = quarter * 32 + lane;   // this lane's key of a tile, and its dim of O
        const uint32_t mx_s = fix_base + C::FIX_MX + grp * 16 * CG;
        const uint32_t f2_s = fix_base + C::FIX_F2 + cb * 4, m_s = fix_base + C::FIX_M + cb * 4;
        bool ok = true;
        int g = 0;
        for (int k = 0;; ++k) {
            const int r = k % kRing;
            ok &= wait_warp(iready + 8 * r, (uint32_t)(k / kRing) & 1u);
            const Unit8 u = read_unit(r);   // all of the group go on, or none: here, or by the vote of the unit's first tile
            if (!ok || u.b < 0) {
                if (bar_any(bar, 128, !ok)) ok = false;
                break;
            }
            const uint32_t oc = tl + C::O_COL + (k & 1) * 3 * RP + cb;   // this unit's O
            const int L = u.P + u.n;
            float2 m[CG / 2], l[CG / 2];   // kBase - reference maximum of exponent + log2(value scale); sums over this lane's keys
#pragma unroll
            for (int c = 0; c < CG / 2; ++c) {
                m[c] = make_float2(1e30f, 1e30f);
                l[c] = make_float2(0.f, 0.f);
            }
            const uint32_t qs = fix_base + C::FIX_QS + (r * 64 + cb) * 4;   // query scales, there before the first scores
            int j = u.j0;
            // y: the columns' exponents before the maximum is taken off; vs: the key's value scale, lv: its log2
            auto scores = [&](float2 (&y)[CG / 2], float &vs, float &lv) {
                const int x = g & 1;
                ok &= wait_warp(sfull + 8 * x, (uint32_t)(g >> 1) & 1u);   // a failure ends the unit with the next vote
                tc_fence_after();
                const uint32_t side = sm_base + C::OFF_SIDE + g % C::STAGES * C::SIDE + kslot * 4;
                float s[CG];
                tc_ldn<CG>(tl + C::S_COL + x * RP + cb, s);
                float ks = lds1(side) * a.scale_log2;
                vs = lds1(side + 512);
                if (!(vs <= 3.402823466e38f)) {   // a poisoned value row: NaN to every row that sees it
                    ks = __int_as_float(0x7fc00000);
                    vs = 0.f;
                }
                lv = lg2(fmaxf(vs, kScaleMin));
                tc_wait_ld();
#pragma unroll
                for (int c = 0; c < CG / 4; ++c) {
                    const float4 v = lds4(qs + 16 * c);
                    const float2 k2 = make_float2(ks, ks);
                    y[2 * c] = __fmul2_rn(__fmul2_rn(make_float2(s[4 * c], s[4 * c + 1]), make_float2(v.x, v.y)), k2);
                    y[2 * c + 1] = __fmul2_rn(__fmul2_rn(make_float2(s[4 * c + 2], s[4 * c + 3]), make_float2(v.z, v.w)), k2);
                }
            };
            auto above = [&](const float2 (&y)[CG / 2], float lv) -> float {   // the furthest above its column's maximum
                float top = -INFINITY, top2 = -INFINITY;
#pragma unroll
                for (int c = 0; c < CG / 2; ++c) {
                    const float2 d = __fadd2_rn(y[c], m[c]);
                    top = fmaxf(top, d.x);
                    top2 = fmaxf(top2, d.y);
                }
                return fmaxf(top, top2) + lv;
            };
            auto write_p = [&](const float2 (&y)[CG / 2], float vs) {
                const float2 rv = make_float2(vs, vs);
                const uint32_t pd = fix_base + C::FIX_P + (g & 1) * C::P_BYTES + kslot * 64;
                const int flip = (kslot >> 1) & 3;
                constexpr int STEP = CG % 16 == 0 ? 16 : 8;
#pragma unroll
                for (int c = 0; c < CG; c += STEP) {
                    uint32_t w[3][STEP / 4];   // the three parts, four columns a word
#pragma unroll
                    for (int i = 0; i < STEP / 4; ++i) {
                        uint32_t h[2], a1[2], a2[2];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int cc = c / 2 + 2 * i + e;
                            const float2 d = __fadd2_rn(y[cc], m[cc]);
                            const float2 pe = make_float2(ex2(d.x), ex2(d.y));
                            l[cc] = __fadd2_rn(l[cc], pe);
                            const float2 pr = __fmul2_rn(pe, rv);
                            h[e] = half2_of(pr.x, pr.y);
                            a1[e] = hsub2(h[e], h[e] & 0xff00ff00u);
                            a2[e] = hsub2(a1[e], a1[e] & 0xff00ff00u) + 0x00800080u;   // half a step: rounded
                        }
                        w[0][i] = __byte_perm(h[0], h[1], 0x7531);
                        w[1][i] = __byte_perm(a1[0], a1[1], 0x7531);
                        w[2][i] = __byte_perm(a2[0], a2[1], 0x7531);
                    }
#pragma unroll
                    for (int e = 0; e < 3; ++e) {
                        const int col = e * RP + cb + c;
                        const uint32_t d = pd + (col >> 6) * C::P_ATOM + ((((col >> 4) & 3) ^ flip) << 4) + (col & 15);
                        if constexpr (STEP == 16) sts4u(d, w[e][0], w[e][1], w[e][2], w[e][3]);
                        else sts2u(d, w[e][0], w[e][1]);
                    }
                }
            };
            auto hand_over = [&]() {
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull + 8 * (g & 1));
            };
            // the common tile: every key seen by every row, no maximum raised; false with nothing done otherwise
            auto plain_tile = [&]() -> bool {
                float2 y[CG / 2];
                float vs, lv;
                scores(y, vs, lv);
                if (bar_any(bar, 128, above(y, lv) > kBase + kOver || !ok)) return false;
                write_p(y, vs);
                hand_over();
                return true;
            };
            // any one tile; false: a wait has failed
            auto any_tile = [&](bool raise) -> bool {
                const int st = g % C::STAGES, key = j * kTileKeys + kslot;
                float2 y[CG / 2];
                float vs, lv;
                scores(y, vs, lv);
                if (j * kTileKeys + kTileKeys > u.P) {   // tree keys, or keys past the end
                    int from = -0x7fffffff, to = 0x7fffffff;   // the columns that see this lane's key
                    if (key >= u.P) {
                        from = to = 0;
                        if (key < L) {
                            from = (key - u.P) * a.G - u.row0 - cb;
                            to = ldsi(sm_base + C::OFF_SIDE + st * C::SIDE + kslot * 4 + 1024) * a.G - u.row0 - cb;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < CG / 2; ++c) {
                        if (!(2 * c >= from && 2 * c < to)) y[c].x = -INFINITY;
                        if (!(2 * c + 1 >= from && 2 * c + 1 < to)) y[c].y = -INFINITY;
                    }
                }
                if (!raise) raise = bar_any(bar, 128, above(y, lv) > kBase + kOver || !ok);
                if (raise) {
                    // new maxima: of each column over the tile, taken where the old one is passed by 2^kOver
                    float t[CG];
#pragma unroll
                    for (int c = 0; c < CG / 2; ++c) {
                        t[2 * c] = warp_max(y[c].x + lv);
                        t[2 * c + 1] = warp_max(y[c].y + lv);
                    }
                    if (lane == 0) {
#pragma unroll
                        for (int c = 0; c < CG; c += 4)
                            sts4u(mx_s + (quarter * CG + c) * 4, __float_as_uint(t[c]), __float_as_uint(t[c + 1]),
                                  __float_as_uint(t[c + 2]), __float_as_uint(t[c + 3]));
                    }
                    if (bar_any(bar, 128, !ok)) {
                        ok = false;
                        return false;
                    }
                    const bool later = j > u.j0;   // O so far is rescaled once the product before this one has landed in it
                    if (gt < CG) {
                        const uint32_t c = mx_s + gt * 4;
                        const float top = fmaxf(fmaxf(lds1(c), lds1(c + 4 * CG)), fmaxf(lds1(c + 8 * CG), lds1(c + 12 * CG)));
                        const float old = later ? lds1(m_s + gt * 4) : 1e30f, nm = top + old > kBase + kOver ? kBase - top : old;
                        sts1(m_s + gt * 4, nm);
                        sts1(f2_s + gt * 4, ex2(0.5f * (nm - old)));   // root of 2^(old maximum - new): the whole may be below fp32's range
                    }
                    bar_sync(bar, 128);
#pragma unroll
                    for (int c = 0; c < CG / 4; ++c) {
                        const float4 v = lds4(m_s + 16 * c);
                        m[2 * c] = make_float2(v.x, v.y);
                        m[2 * c + 1] = make_float2(v.z, v.w);
                        if (later) {
                            const float4 f = lds4(f2_s + 16 * c);
                            l[2 * c] = __fmul2_rn(__fmul2_rn(l[2 * c], make_float2(f.x, f.y)), make_float2(f.x, f.y));
                            l[2 * c + 1] = __fmul2_rn(__fmul2_rn(l[2 * c + 1], make_float2(f.z, f.w)), make_float2(f.z, f.w));
                        }
                    }
                    if (later) {
                        if (ok && !wait_warp(pvdone + 8 * ((g - 1) & 1), (uint32_t)((g - 1) >> 1) & 1u)) ok = false;
                        tc_fence_after();
                        if (ok && quarter * 32 < D) {
#pragma unroll 1
                            for (int c = 0; c < 3 * CG; c += 4) {
                                float o[4];
                                const uint32_t at = oc + c / CG * RP + c % CG;
                                const float4 f = lds4(f2_s + c % CG * 4);
                                tc_ld4(at, o);
                                tc_wait_ld();
                                o[0] *= f.x * f.x;
                                o[1] *= f.y * f.y;
                                o[2] *= f.z * f.z;
                                o[3] *= f.w * f.w;
                                tc_st4(at, o);
                            }
                            tc_wait_st();
                        }
                    }
                }
                write_p(y, vs);
                if (j * kTileKeys + kTileKeys > L && ok) {
                    // V's rows past the last key may hold anything: zeros (whose weights are zero too)
                    const uint32_t vt = sm_base + st * C::STAGE_BYTES + C::OP_BYTES;
                    const int r0 = (L - j * kTileKeys) * (D / 16);
#pragma unroll 1
                    for (int i = r0 + tid - 128; i < kTileKeys * (D / 16); i += 32 * C::SM_WARPS)
                        sts4u(vt + i * 16, 0u, 0u, 0u, 0u);
                }
                hand_over();
                return true;
            };
            const int plain_end = min(u.j1, u.P / kTileKeys);   // tiles before the first with tree keys
            bool gone = false;
            while (j < u.j1) {
                bool raise = j == u.j0;
                if (!raise) {
#pragma unroll 1
                    while (j < plain_end && plain_tile()) {
                        ++j;
                        ++g;
                    }
                    if (j == u.j1) break;
                    raise = j < plain_end;
                }
                if (!any_tile(raise)) {
                    gone = true;
                    break;
                }
                ++j;
                ++g;
            }
            if (gone) break;
            // the unit's sums and maxima to the output warps, once those of two units before are read
            float v[CG];
#pragma unroll
            for (int c = 0; c < CG / 2; ++c) {
                v[2 * c] = l[c].x;
                v[2 * c + 1] = l[c].y;
            }
            if (k >= 2) ok &= wait_warp(ofree + 8 * (k & 1), (uint32_t)(k / 2 - 1) & 1u);
            reduce_scatter<CG>(v, lane);
            const uint32_t sum = fix_base + C::FIX_SUM + (k & 1) * C::SUM_BYTES;
            if (lane % (32 / CG) == 0) sts1(sum + (quarter * 64 + cb + lane / (32 / CG)) * 4, v[0]);
            if (gt < CG) sts1(sum + (4 * 64 + cb + gt) * 4, -lds1(m_s + gt * 4));
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(sumfull + 8 * (k & 1));
                mbar_arrive(ifree + 8 * r);
            }
        }
        if (!ok) misc[1] = 1;
    } else {   // -------------------------------------------------------- query rows, output
        if constexpr (C::SPLIT) take_registers<false, C::OTHER_REGS>();
        // Unit k's query rows are split here, then unit k - 1 is written out: its last product, its writing and the
        // next unit's first scores run at the same time.
        const int quarter = warp & 3, dim = quarter * 32 + lane;
        bool ok = true;
        for (int k = 0;; ++k) {
            const int r = k % kRing;
            if (!wait_warp(iready + 8 * r, (uint32_t)(k / kRing) & 1u)) ok = false;
            if (bar_any(15, 128, !ok)) {   // all four warps go on, or none
                ok = false;
                break;
            }
            const bool more = ldsi(fix_base + C::FIX_INFO + r * 48) >= 0;
            if (more) {
                if (!wait_warp(qraw + 8 * (k & 1), (uint32_t)(k >> 1) & 1u)) ok = false;
                const uint32_t qd = fix_base + C::FIX_Q + (k & 1) * C::Q_BYTES;
                constexpr int LPR = 8, EPL = D / LPR;   // lanes of a row; values of a lane
                const int sub = lane % LPR;
#pragma unroll 1
                for (int c = quarter * (RP / 4) + lane / LPR; c < (quarter + 1) * (RP / 4); c += 4) {
                    uint32_t w[EPL / 2];   // two values each
                    const uint32_t src = qd + ((sub >= LPR / 2 ? RP : 0) + c) * D + sub % (LPR / 2) * (2 * EPL);
#pragma unroll
                    for (int e = 0; e < EPL / 2; e += 2)
                        asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[e]), "=r"(w[e + 1]) : "r"(src + 4 * e) : "memory");
                    uint32_t top = 0;   // two |values| at a time, which order as their bits do, infinities and NaN on top
#pragma unroll
                    for (int e = 0; e < EPL / 2; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
#pragma unroll
                    for (int o = LPR / 2; o; o >>= 1) top = __vmaxu2(top, __shfl_xor_sync(~0u, top, o));
                    top = max(top >> 16, top & 0xffffu);
                    // 2^(exponent - 7), within the normal numbers whose reciprocal is one too
                    int ex = (int)(top >> 7) - 7;
                    ex = ex < 4 ? 4 : ex;
                    const float inv = __uint_as_float((uint32_t)(254 - ex) << 23);
#pragma unroll
                    for (int e = 0; e < EPL / 4; ++e) {
                        uint32_t h2[2], l2[2];
#pragma unroll
                        for (int f = 0; f < 2; ++f) {   // fp16 holds the scaled values and every difference here
                            const uint32_t v = w[2 * e + f];
                            const float2 y = __fmul2_rn(make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)),
                                                        make_float2(inv, inv));
                            const uint32_t y16 = half2_of(y.x, y.y);
                            h2[f] = half2_to_fp8x2(y16);
                            l2[f] = half2_to_fp8x2(hsub2(y16, fp8x2_to_half2(h2[f])));
                        }
                        // 16-byte chunks of a row are permuted as the MMA's descriptor says
                        const int at = sub * EPL + 4 * e;
                        auto place = [&](int row) {
                            const int flip = D == 128 ? row & 7 : (row >> 1) & 3;
                            return qd + row * D + (((at >> 4) ^ flip) << 4) + (at & 15);
                        };
                        stsi(place(c), (int)(h2[0] | h2[1] << 16));
                        stsi(place(RP + c), (int)(l2[0] | l2[1] << 16));
                    }
                    if (sub == 0) {
                        const int scale = top >= 0x7f80u ? 0x7fc00000 : (int)((uint32_t)ex << 23);
                        stsi(fix_base + C::FIX_QS + (r * 64 + c) * 4, scale);
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(qready + 8 * (k & 1));
            }
            if (k > 0) {
                const int par = (k - 1) & 1, dr = (k - 1) % kRing;
                const Unit8 done = read_unit(dr);
                if (ok && (!wait_warp(sumfull + 8 * par, (uint32_t)((k - 1) >> 1) & 1u) ||
                           !wait_warp(odone + 8 * par, (uint32_t)((k - 1) >> 1) & 1u)))
                    ok = false;
                if (bar_any(15, 128, !ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // lane c: factor and place of columns c and 32 + c; a part keeps its own maximum and sum, a whole
                // unit is divided by its sum
                float f[2] = {0.f, 0.f};
                int place[2] = {-1, -1};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = h * 32 + lane;
                    if (c < RP) {
                        const uint32_t sum = fix_base + C::FIX_SUM + par * C::SUM_BYTES + c * 4;
                        const float lsum = (lds1(sum) + lds1(sum + 256)) + (lds1(sum + 512) + lds1(sum + 768));
                        f[h] = done.parts > 1 ? 1.f : 1.f / lsum;
                        place[h] = ldsi(fix_base + C::FIX_QROW + (dr * 64 + c) * 4);
                        if (done.parts > 1 && quarter == 0)
                            a.part_ml[(size_t)(done.slot + done.part) * RP + c] = make_float2(lds1(sum + 1024), lsum);
                    }
                }
                __nv_bfloat16 *ob = a.out + (size_t)done.b * n_max * a.Hq * D;
                const uint32_t oc = tmem + ((uint32_t)(quarter * 32) << 16) + C::O_COL + par * 3 * RP;
                if (quarter * 32 < D) {
#pragma unroll 1
                    for (int c = 0; c < RP; c += 4) {
                        float o[3][4];
#pragma unroll
                        for (int i = 0; i < 3; ++i) tc_ld4(oc + i * RP + c, o[i]);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[0][e] = ((o[0][e] + o[1][e]) + o[2][e]) * __shfl_sync(~0u, c < 32 ? f[0] : f[1], (c + e) & 31);
                        if (done.parts > 1) {
                            float *po = a.part_o + ((size_t)(done.slot + done.part) * RP + c) * D + dim;
#pragma unroll
                            for (int e = 0; e < 4; ++e) po[e * D] = o[0][e];
                        } else {
                            // two columns at a time: even lanes store dims (d, d + 1) of the first, odd lanes of the second
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                const float keep = lane & 1 ? o[0][e + 1] : o[0][e], send = lane & 1 ? o[0][e] : o[0][e + 1];
                                const float got = __shfl_xor_sync(~0u, send, 1);
                                const int row = __shfl_sync(~0u, c < 32 ? place[0] : place[1], (c + e + (lane & 1)) & 31);
                                const __nv_bfloat162 v = lane & 1 ? __floats2bfloat162_rn(got, keep) : __floats2bfloat162_rn(keep, got);
                                if (row >= 0) *(__nv_bfloat162 *)(ob + (size_t)row * D + (dim & ~1)) = v;
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ofree + 8 * par);
                if (done.parts > 1) {   // the last part of the item to finish joins them
                    __threadfence();
                    bar_sync(15, 128);
                    if (quarter == 0 && lane == 0) {
                        unsigned *cnt = a.joins + done.slot;
                        const bool last = atomicAdd(cnt, 1u) == (unsigned)done.parts - 1;
                        if (last) *cnt = 0u;
                        misc[3] = last;
                    }
                    bar_sync(15, 128);
                    if (misc[3])
                        join_parts<D, RP>(a.part_ml + (size_t)done.slot * RP, a.part_o + (size_t)done.slot * RP * D, done.parts,
                                          fix_base + C::FIX_QROW + dr * 256, ob);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(ifree + 8 * dr);
            }
            if (!more) break;
        }
        if (!ok && lane == 0) misc[1] = 1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
    if (tid == 0) {
        if (misc[1]) flag(a.status, TS_STATUS_TIMEOUT);
        // the last CTA returns the queue to zero: every CTA counted here has stopped taking units
        __threadfence();
        if (atomicAdd(a.queue + 1, 1u) == gridDim.x - 1) {
            a.queue[0] = 0u;
            a.queue[1] = 0u;
        }
    }
}

// ------------------------------------------------------------------ plan ---
struct Plan8 {
    int rp, blocks, slots;
    size_t ml, o, bytes;   // offsets of the parts, all bytes
};

// RP: the rows there can be, cut into equal blocks of at most 64, rounded up to
// 16. Slots: no more than there can be parts. The counters (queue, joins) lie
// ahead of every size's parts, so that one workspace serves calls of any sizes
// it is large enough for, one after another.
Plan8 plan8(int B, int Hkv, int G, int n_max, int d) {
    Plan8 p;
    const long long rows = (long long)n_max * G;
    p.blocks = (int)((rows + 63) / 64);
    p.rp = (int)(((rows + p.blocks - 1) / p.blocks + 15) / 16 * 16);
    p.blocks = (int)((rows + p.rp - 1) / p.rp);
    const long long most = (long long)B * Hkv * p.blocks * kMaxCuts;
    p.slots = B > kReqCache ? 0 : (int)(most < kSlotsPerSm * num_sms() ? most : kSlotsPerSm * num_sms());
    size_t at = 256 + ((size_t)kSlotsPerSm * num_sms() * sizeof(unsigned) + 255) / 256 * 256;
    p.ml = at;
    at += (size_t)p.slots * p.rp * sizeof(float2);
    p.o = (at + 255) / 256 * 256;
    p.bytes = p.o + (size_t)p.slots * p.rp * d * sizeof(float);
    return p;
}

// Rows of d codes; boxes of box_rows whole rows, swizzled by the row's width.
bool make_map8(CUtensorMap *map, const void *base, int d, long long rows, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)d};
    cuuint32_t box[2] = {(cuuint32_t)d, (cuuint32_t)box_rows}, estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int RP>
cudaError_t launch8(const CUtensorMap &mk, const CUtensorMap &mv, const Attn8Args &a, int grid, cudaStream_t s,
                    const char **why) {
    using C = Cfg8<D, RP>;
    cudaError_t e = cudaFuncSetAttribute(k_attn_kv8<D, RP>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (C::SPLIT) {   // the kernel waits for registers that a smaller launch would not have
        cudaFuncAttributes at;
        if ((e = cudaFuncGetAttributes(&at, k_attn_kv8<D, RP>)) != cudaSuccess) return e;
        if ((at.numRegs + 7) / 8 * 8 < C::LAUNCH_REGS) {   // given out in eights
            *why = "this build's kernel has fewer registers a thread than its warps hand to one another";
            return cudaErrorInvalidConfiguration;
        }
    }
    return launch(k_attn_kv8<D, RP>, dim3(grid), dim3(C::THREADS), C::SMEM, s, mk, mv, a);
}

}  // namespace

size_t kv8_attention_ws_bytes(int B, int Hq, int Hkv, int n_max, int d, int) {
    return plan8(B, Hkv, Hq / Hkv, n_max, d).bytes;
}

cudaError_t launch_attn_kv8(void *out, const void *q, const ts_kv8 &kv, int Hq, const int32_t *prefix_len,
                            const ts_tree &t, float scale, void *ws, uint32_t *status, cudaStream_t s,
                            const char **why) {
    const int G = Hq / kv.H;
    const Plan8 p = plan8(t.B, kv.H, G, t.n_max, kv.d);
    const bool paged = kv.block_table != nullptr;
    const long long rows = paged ? (long long)kv.num_pages * kv.H * TS_PAGE_KEYS : (long long)kv.B * kv.H * kv.L_max;
    CUtensorMap mk, mv;
    if (!make_map8(&mk, kv.k, kv.d, rows, paged ? TS_PAGE_KEYS : kTileKeys) ||
        !make_map8(&mv, kv.v, kv.d, rows, paged ? TS_PAGE_KEYS : kTileKeys)) {
        *why = "cuTensorMapEncodeTiled failed for the 8-bit cache";
        return cudaErrorInvalidValue;
    }
    unsigned char *w = (unsigned char *)ws;
    Attn8Args a = {(__nv_bfloat16 *)out, (const __nv_bfloat16 *)q, kv.k_scale, kv.v_scale, prefix_len, t, Hq, kv.H, G,
                   kv8_rows(kv), scale * kLog2e, kv8_pages(kv), status, (unsigned *)w,
                   (unsigned *)(w + 256), (float2 *)(w + p.ml), (float *)(w + p.o), p.slots};
    // no more CTAs than there can be units
    const long long tiles = (a.rows + kTileKeys - 1) / kTileKeys, cuts = (tiles + kMinCut - 1) / kMinCut;
    const long long units = (long long)t.B * kv.H * p.blocks * (p.slots ? (cuts < kMaxCuts ? cuts : kMaxCuts) : 1);
    const int grid = (int)(units < num_sms() ? units : num_sms());
    if (kv.d == 128) switch (p.rp) {
        case 16: return launch8<128, 16>(mk, mv, a, grid, s, why);
        case 32: return launch8<128, 32>(mk, mv, a, grid, s, why);
        case 48: return launch8<128, 48>(mk, mv, a, grid, s, why);
        default: return launch8<128, 64>(mk, mv, a, grid, s, why);
    }
    switch (p.rp) {
        case 16: return launch8<64, 16>(mk, mv, a, grid, s, why);
        case 32: return launch8<64, 32>(mk, mv, a, grid, s, why);
        case 48: return launch8<64, 48>(mk, mv, a, grid, s, why);
        default: return launch8<64, 64>(mk, mv, a, grid, s, why);
    }
}

}  // namespace ts
