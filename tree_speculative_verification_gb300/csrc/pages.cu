// pages.cu -- a paged cache's housekeeping: pages to requests that grow and
// back from those that shrink, the slot of every new row, and K/V rows into
// their slots.
#include <algorithm>

#include "decode.cuh"

namespace ts {
namespace {

// ---------------------------------------------------------- pages and slots ----
// One launch, in which no CTA waits for another: a request's pages follow from
// running sums over the lengths, which every CTA forms for itself (three sums
// of B integers from L2), and a new row's page is read where it comes from, the
// request's own table entry or the ring of free pages, never where another CTA
// writes it. The pages that come back go behind the ring's free part, so that
// no entry is both read and written. What the call changes in place (pages
// held, the ring's head and count) is written by the CTA that ends last.
//
// Integers; bound by the chain of loads (lengths, then table or ring entries)
// up to some 100k rows, then by the 4 bytes a row.
constexpr int kPageThreads = 512;

struct PageArgs {
    ts_page_pool pool;
    int32_t *new_held, *new_state, *slot, *slot_offset;
    const int32_t *row_begin, *row_end;
    int max_slots, per_cta;   // per_cta: slots of a CTA, a multiple of 4
    bool slot_vec;            // slot is 16-byte aligned
    uint32_t *status;
};

struct Sums {
    long long n, take, back;   // rows, pages taken, pages given back
};

// Inclusive running sums over the CTA's threads. part: one entry a warp.
__device__ Sums block_sums(Sums v, Sums *part) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long n = __shfl_up_sync(~0u, v.n, o), t = __shfl_up_sync(~0u, v.take, o),
                        r = __shfl_up_sync(~0u, v.back, o);
        if (lane >= o) v.n += n, v.take += t, v.back += r;
    }
    __syncthreads();   // part may still be read
    if (lane == 31) part[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v.n += part[w].n, v.take += part[w].take, v.back += part[w].back;
    return v;
}

struct Request {
    int held, begin;
    long long want;   // pages of its rows
    Sums own;
    bool sound;       // its lengths are
};

__device__ Request request(const PageArgs &a, int b) {
    Request r = {};
    if (b >= a.pool.B) return r;
    const int end = a.row_end[b];
    r.held = a.pool.held[b];
    r.begin = a.row_begin ? a.row_begin[b] : end;
    r.own.n = max(0LL, (long long)end - r.begin);
    r.want = ((long long)end + TS_PAGE_KEYS - 1) / TS_PAGE_KEYS;
    r.sound = r.begin >= 0 && r.begin <= end && r.want <= a.pool.max_pages && r.held >= 0 && r.held <= a.pool.max_pages;
    if (r.sound) r.own.take = max(0LL, r.want - r.held), r.own.back = max(0LL, r.held - r.want);
    return r;
}

// Entry k of the ring, k counted from its start and below three times round.
__device__ __forceinline__ int ring_at(long long k, int num) {
    k -= k >= num ? num : 0;
    return (int)(k - (k >= num ? num : 0));
}

// n ids from one place to another, by a warp: four loads under way a lane.
template <typename From, typename To>
__device__ __forceinline__ void move_ids(int n, From from, To to) {
    for (int i = threadIdx.x & 31; i < n; i += 128) {
        int id[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + 32 * k < n) id[k] = *from(i + 32 * k);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (i + 32 * k < n) *to(i + 32 * k) = id[k];
    }
}

__global__ void __launch_bounds__(kPageThreads) k_pages_build(PageArgs a) {
    __shared__ Sums part[kPageThreads / 32];
    __shared__ long long off_s[kPageThreads + 1];   // first slots of the tile's requests, and the tile's end
    __shared__ int begin_s[kPageThreads], held_s[kPageThreads], want_s[kPageThreads], from_s[kPageThreads];
    __shared__ bool ok_s[kPageThreads];
    __shared__ unsigned long long taken_s;
    __shared__ int last_s;
    const int tid = threadIdx.x, B = a.pool.B, num = a.pool.num_pages, width = a.pool.max_pages;
    int32_t *const ring = a.pool.ring, *const table = a.pool.block_table;
    pdl_wait();
    pdl_trigger();
    const int head = a.pool.ring_state[0], count = a.pool.ring_state[1];
    // what comes back in all: with it the ring must not hold more than the pool's pages
    Request r = request(a, tid);
    Sums all = r.own;
    for (int b = tid + kPageThreads; b < B; b += kPageThreads) {
        const Request x = request(a, b);
        all.n += x.own.n, all.take += x.own.take, all.back += x.own.back;
    }
    if (tid == 0) taken_s = 0;
    all = block_sums(all, part);
    __syncthreads();
    if (tid == kPageThreads - 1) part[0] = all;
    __syncthreads();
    all = part[0];
    const bool pool_ok = head >= 0 && head < num && count >= 0 && count + all.back <= num;
    const long long s0 = min((long long)blockIdx.x * a.per_cta, (long long)a.max_slots),
                    s1 = min(s0 + a.per_cta, (long long)a.max_slots);
    uint32_t bits = 0;
    if (!pool_ok || (a.slot && all.n > a.max_slots)) bits |= TS_STATUS_INDEX;

    Sums at = {};
    for (int base = 0; base < B; base += kPageThreads) {   // a tile of requests, a thread each
        const int b = base + tid;
        if (base) r = request(a, b);
        const Sums run = block_sums(r.own, part);
        const long long first = at.n + run.n - r.own.n, from = at.take + run.take - r.own.take;
        const bool ok = b < B && pool_ok && r.sound && (r.own.take == 0 || from + r.own.take <= count);
        if (b < B && !r.sound) bits |= TS_STATUS_INDEX;
        if (b < B && pool_ok && r.sound && !ok) bits |= TS_STATUS_NO_PAGES;
        if (ok && r.own.take) atomicMax(&taken_s, (unsigned long long)(from + r.own.take));
        off_s[tid] = first, begin_s[tid] = r.begin, held_s[tid] = r.held, ok_s[tid] = ok;
        want_s[tid] = r.sound ? (int)r.want : r.held;
        // a request takes or gives back: where its first page comes from, or goes behind the ring's free part
        from_s[tid] = !ok ? 0 : ring_at(head + (r.own.take ? from : count + at.back + run.back - r.own.back), num);
        if (tid == kPageThreads - 1) off_s[kPageThreads] = first + r.own.n;
        if (blockIdx.x == 0 && b < B && a.slot_offset) {
            a.slot_offset[b] = (int)min(first, (long long)INT32_MAX);
            if (b == B - 1) a.slot_offset[B] = (int)min(first + r.own.n, (long long)INT32_MAX);
        }
        __syncthreads();
        for (int i = tid >> 5; i < min(kPageThreads, B - base); i += kPageThreads / 32) {   // a warp a request
            if ((base + i) % gridDim.x != blockIdx.x || !ok_s[i]) continue;
            const int held = held_s[i], want = want_s[i], from_i = from_s[i];
            int32_t *const row = table + (size_t)(base + i) * width;
            auto in_ring = [&](int k) { return ring + ring_at((long long)from_i + k, num); };
            move_ids(want - held, in_ring, [&](int k) { return row + held + k; });
            move_ids(held - want, [&](int k) { return row + want + k; }, in_ring);
        }
        if (a.slot) {   // the tile's slots in this CTA's range, four a thread
            const long long lo = max(s0, off_s[0]), hi = min(s1, off_s[kPageThreads]);
            for (long long i0 = (lo & ~3LL) + 4 * tid; i0 < hi; i0 += 4 * kPageThreads) {
                const long long i1 = max(i0, lo);
                int x = 0, y = kPageThreads - 1, v[4];   // the last request whose first slot is not behind i1
                while (x < y) {
                    const int m = (x + y + 1) >> 1;
                    if (off_s[m] <= i1) x = m;
                    else y = m - 1;
                }
                int page = -1, p_now = -1;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const long long i = i0 + e;
                    v[e] = -1;
                    if (i < lo || i >= hi) continue;
                    while (off_s[x + 1] <= i) ++x, p_now = -1;
                    if (!ok_s[x]) continue;
                    const int j = begin_s[x] + (int)(i - off_s[x]), p = j / TS_PAGE_KEYS;
                    if (p != p_now) {
                        p_now = p;
                        page = p < held_s[x] ? table[(size_t)(base + x) * width + p]
                                             : ring[ring_at((long long)from_s[x] + (p - held_s[x]), num)];
                        if (page < 0 || page >= num) page = -1, bits |= TS_STATUS_INDEX;
                    }
                    if (page >= 0) v[e] = page * TS_PAGE_KEYS + j % TS_PAGE_KEYS;
                }
                if (a.slot_vec && i0 >= lo && i0 + 4 <= hi)
                    *reinterpret_cast<int4 *>(a.slot + i0) = make_int4(v[0], v[1], v[2], v[3]);
                else
                    for (int e = 0; e < 4; ++e)
                        if (i0 + e >= lo && i0 + e < hi) a.slot[i0 + e] = v[e];
            }
        }
        __syncthreads();
        if (tid == kPageThreads - 1) part[0] = run;
        __syncthreads();
        at.n += part[0].n, at.take += part[0].take, at.back += part[0].back;
    }
    if (a.slot)
        for (long long i = max(s0, at.n) + tid; i < s1; i += kPageThreads) a.slot[i] = -1;
    if (bits) flag(a.status, bits);

    // the last CTA to come here: every other one has read what is now written
    __syncthreads();
    if (tid == 0) {
        last_s = gridDim.x == 1;
        if (gridDim.x > 1) {
            __threadfence();
            unsigned *done = (unsigned *)a.pool.ring_state + 2;
            last_s = atomicAdd(done, 1u) == gridDim.x - 1;
            if (last_s) *done = 0;
            __threadfence();
        }
    }
    __syncthreads();
    if (!last_s) return;
    long long take = 0;
    for (int base = 0; base < B; base += kPageThreads) {
        const int b = base + tid;
        if (B > kPageThreads) r = request(a, b);
        const Sums run = block_sums(r.own, part);
        if (b < B) {
            const bool ok = pool_ok && r.sound && (r.own.take == 0 || take + run.take <= count);
            a.new_held[b] = ok ? (int)r.want : r.held;
        }
        __syncthreads();
        if (tid == kPageThreads - 1) part[0] = run;
        __syncthreads();
        take += part[0].take;
    }
    if (tid == 0) {
        const long long taken = (long long)taken_s;
        a.new_state[0] = pool_ok ? (int)((head + taken) % num) : head;
        a.new_state[1] = pool_ok ? (int)(count - taken + all.back) : count;
    }
}

// --------------------------------------------------------------- rows by slot ----
// cache[slot / 64][h][slot % 64] = new[t][h]: 16-byte pieces, a CTA a few
// tokens, the new rows' loads under way before their slots are known.
constexpr int kSlotThreads = 256;

template <int TB>
__global__ void __launch_bounds__(kSlotThreads) k_append_slots(uint4 *k_pages, uint4 *v_pages, const uint4 *k_new,
                                                               const uint4 *v_new, long long k_stride,
                                                               long long v_stride, const int32_t *slot, int T, int H,
                                                               int vec_log2, int num_pages, uint32_t *status) {
    pdl_wait();
    pdl_trigger();
    const int t0 = blockIdx.x * TB, per = H << vec_log2;
    for (int p = threadIdx.x; p < per; p += kSlotThreads) {
        uint4 k[TB], v[TB];
        int at[TB];
#pragma unroll
        for (int i = 0; i < TB; ++i)
            if (t0 + i < T) {
                at[i] = slot[t0 + i];
                k[i] = __ldcs(k_new + (t0 + i) * k_stride + p);
                v[i] = __ldcs(v_new + (t0 + i) * v_stride + p);
            }
        const int h = p >> vec_log2, c = p & ((1 << vec_log2) - 1);
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            if (t0 + i >= T || at[i] < 0) {
                if (t0 + i < T && at[i] < -1 && p == 0) flag(status, TS_STATUS_INDEX);
                continue;
            }
            const int page = at[i] / TS_PAGE_KEYS, row = at[i] % TS_PAGE_KEYS;
            if (page >= num_pages) {
                if (p == 0) flag(status, TS_STATUS_INDEX);
                continue;
            }
            const size_t dst = ((((size_t)page * H + h) * TS_PAGE_KEYS + row) << vec_log2) + c;
            k_pages[dst] = k[i];
            v_pages[dst] = v[i];
        }
    }
}

}  // namespace

cudaError_t launch_pages_build(const ts_page_pool &pool, int32_t *new_held, int32_t *new_state, int32_t *slot,
                               int max_slots, int32_t *slot_offset, const int32_t *row_begin, const int32_t *row_end,
                               uint32_t *status, cudaStream_t s) {
    PageArgs a{pool, new_held, new_state, slot, slot_offset, row_begin, row_end, slot ? max_slots : 0, 0,
               ((uintptr_t)slot & 15) == 0, status};
    const int ctas = (int)std::min<long long>(2LL * num_sms(), 1 + (long long)a.max_slots / (8 * kPageThreads));
    a.per_cta = ((a.max_slots + ctas - 1) / ctas + 3) / 4 * 4;
    return launch(k_pages_build, dim3(ctas), dim3(kPageThreads), 0, s, a);
}

cudaError_t launch_append_slots(const ts_paged_kv &kv, const void *k_new, const void *v_new, long long k_stride,
                                long long v_stride, const int32_t *slot, int T, int H, int d, uint32_t *status,
                                cudaStream_t s) {
    const int vec_log2 = d == 128 ? 4 : 3;
    auto go = [&](auto kern, int tb) {
        return launch(kern, dim3((T + tb - 1) / tb), dim3(kSlotThreads), 0, s, (uint4 *)kv.k_pages, (uint4 *)kv.v_pages,
                      (const uint4 *)k_new, (const uint4 *)v_new, k_stride / 8, v_stride / 8, slot, T, H, vec_log2,
                      (int)kv.num_pages, status);
    };
    return T > 1024 ? go(k_append_slots<4>, 4) : go(k_append_slots<1>, 1);
}

}  // namespace ts
