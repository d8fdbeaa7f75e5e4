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
// Integers; bound by the chain of loads (lengths, then table or ring entries):
// 8 requests 4.6 us. 2.1 M rows of 256 requests take 12 us, where a write of their
// slots alone would take 1.4: the sums and searches that every CTA makes for
// itself (issue slots 60%), and the last CTA's turn.
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
__device__ __forceinline__ int ring_at(int k, int num) {
    k -= k >= num ? num : 0;
    return k - (k >= num ? num : 0);
}

// Of 2 `most` rising numbers (a power of two) the last one that is i or less (the first is).
__device__ __forceinline__ int last_upto(const int *s, int most, int i) {
    int x = 0;
    for (int step = most; step; step /= 2)
        if (s[x + step] <= i) x += step;
    return x;
}

__device__ __forceinline__ int clamped(long long v) { return (int)min(v, (long long)INT32_MAX); }

// Rows, pages taken and pages given back each stand in one line, the requests' one after the other; every CTA takes an equal
// stretch of each line and finds a stretch's requests by the running sums.
__global__ void __launch_bounds__(kPageThreads, 2) k_pages_build(PageArgs a) {
    __shared__ Sums part[kPageThreads / 32], all_s, tile_s;
    __shared__ int row_s[kPageThreads + 1], take_s[kPageThreads + 1], back_s[kPageThreads + 1];   // a tile's requests' first ones
    __shared__ int begin_s[kPageThreads], held_s[kPageThreads], want_s[kPageThreads];
    __shared__ bool ok_s[kPageThreads];
    __shared__ int taken_s, last_s;
    const int tid = threadIdx.x, B = a.pool.B, num = a.pool.num_pages, width = a.pool.max_pages;
    int32_t *const ring = a.pool.ring, *const table = a.pool.block_table;
    pdl_wait();
    pdl_trigger();
    const int head = a.pool.ring_state[0], count = a.pool.ring_state[1];
    Request r = request(a, tid);
    if (tid == 0) taken_s = 0;
    // running sums over the first tile; of all requests (what comes back must not fill the ring beyond the pool's pages)
    Sums run = block_sums(r.own, part), all = run;
    if (B > kPageThreads) {
        Sums more = r.own;
        for (int b = tid + kPageThreads; b < B; b += kPageThreads) {
            const Request x = request(a, b);
            more.n += x.own.n, more.take += x.own.take, more.back += x.own.back;
        }
        all = block_sums(more, part);
    }
    if (tid == kPageThreads - 1) all_s = all;
    __syncthreads();
    all = all_s;
    const bool pool_ok = head >= 0 && head < num && count >= 0 && count + all.back <= num;
    uint32_t bits = 0;
    if (!pool_ok || (a.slot && all.n > a.max_slots)) bits |= TS_STATUS_INDEX;
    // the CTA's stretches
    const int c = blockIdx.x, ctas = gridDim.x;
    const int s0 = (int)min((long long)c * a.per_cta, (long long)a.max_slots), s1 = (int)min((long long)s0 + a.per_cta, (long long)a.max_slots);
    const int takes = (int)min(all.take, (long long)max(count, 0)), t_per = (takes + ctas - 1) / ctas, b_per = ((int)min(all.back, (long long)num) + ctas - 1) / ctas;

    Sums at = {};
    bool ok = false;
    for (int base = 0; base < B; base += kPageThreads) {   // a tile of requests, a thread each
        const int b = base + tid;
        if (base) {
            r = request(a, b);
            run = block_sums(r.own, part);
        }
        const long long first = at.n + run.n - r.own.n, from = at.take + run.take - r.own.take;
        ok = b < B && pool_ok && r.sound && (r.own.take == 0 || from + r.own.take <= count);
        if (b < B && !r.sound) bits |= TS_STATUS_INDEX;
        if (b < B && pool_ok && r.sound && !ok) bits |= TS_STATUS_NO_PAGES;
        const int served = __reduce_max_sync(~0u, ok && r.own.take ? (int)(from + r.own.take) : 0);   // of the line; rises from warp to warp
        if ((tid & 31) == 0 && served) atomicMax(&taken_s, served);
        row_s[tid] = clamped(first), take_s[tid] = clamped(from), back_s[tid] = clamped(at.back + run.back - r.own.back);
        begin_s[tid] = r.begin, held_s[tid] = r.held, want_s[tid] = r.sound ? (int)r.want : r.held, ok_s[tid] = ok;
        if (tid == kPageThreads - 1) {
            row_s[kPageThreads] = clamped(first + r.own.n), take_s[kPageThreads] = clamped(from + r.own.take);
            back_s[kPageThreads] = clamped(at.back + run.back);
            tile_s = run;
        }
        if (c == 0 && b < B && a.slot_offset) {
            a.slot_offset[b] = clamped(first);
            if (b == B - 1) a.slot_offset[B] = clamped(first + r.own.n);
        }
        __syncthreads();
        const Sums tile = tile_s;
        const int most = B - base > 1 ? 1 << (31 - __clz(min(B - base, kPageThreads) - 1)) : 1;   // half of the tile's requests' number, rounded up
        // Pages taken: as many of the line as are served, which are whole requests; and pages given back, behind the ring's free
        // part. A thread's first ones are read before anything is written.
        const int t1 = pool_ok ? min(min(take_s[kPageThreads], taken_s), (c + 1) * t_per) : 0,
                  b1 = pool_ok ? min(back_s[kPageThreads], (c + 1) * b_per) : 0;
        int ti = max(take_s[0], c * t_per) + tid, bi = max(back_s[0], c * b_per) + tid;
        auto move = [&] {
            while (ti < t1 || bi < b1) {
                int t_page = 0, b_page = 0, *t_to = nullptr;
                if (ti < t1) {
                    const int x = last_upto(take_s, most, ti);
                    t_page = ring[ring_at(head + ti, num)];
                    t_to = &table[(size_t)(base + x) * width + held_s[x] + (ti - take_s[x])];
                }
                if (bi < b1) {
                    const int x = last_upto(back_s, most, bi);
                    b_page = table[(size_t)(base + x) * width + want_s[x] + (bi - back_s[x])];
                }
                if (ti < t1) *t_to = t_page;
                if (bi < b1) ring[ring_at(head + count + bi, num)] = b_page;
                ti += kPageThreads, bi += kPageThreads;
            }
        };
        if (a.slot) {   // slots, four a thread
            const int lo = max(s0, row_s[0]), hi = min(s1, row_s[kPageThreads]);
            // page p of the tile's request x: its own, or the ring's where it is taken only now
            auto page_of = [&](int x, int p) {
                return p < held_s[x] ? table[(size_t)(base + x) * width + p] : ring[ring_at(head + take_s[x] + (p - held_s[x]), num)];
            };
            int now = -1;   // the request of the slots before: the next ones' are mostly its
            for (long long i0 = (lo & ~3LL) + 4 * tid; i0 < hi; i0 += 4 * kPageThreads) {
                // Four rows of one request are in one page or two, and their first one's place is enough; of several requests
                // every row has a page of its own (-1: there is none to read).
                int at[4] = {-1, -1, -1, -1}, page[4] = {}, v[4];
                const int i = max((int)i0, lo);
                if (now < 0 || i >= row_s[now + 1]) now = last_upto(row_s, most, i);
                const bool one = i0 >= lo && i0 + 4 <= min(hi, row_s[now + 1]);
                if (one) {
                    if (ok_s[now]) {
                        const int j = begin_s[now] + (i - row_s[now]);
                        at[0] = j % TS_PAGE_KEYS;
                        page[0] = page_of(now, j / TS_PAGE_KEYS);
                        if (at[0] > TS_PAGE_KEYS - 4) page[1] = page_of(now, j / TS_PAGE_KEYS + 1);
                    }
                } else {
                    int y = now;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (i0 + e < lo || i0 + e >= hi) continue;
                        while (row_s[y + 1] <= i0 + e) ++y;
                        if (!ok_s[y]) continue;
                        const int j = begin_s[y] + ((int)i0 + e - row_s[y]);
                        at[e] = j % TS_PAGE_KEYS;
                        page[e] = page_of(y, j / TS_PAGE_KEYS);
                    }
                }
                move();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = one && at[0] >= 0 ? at[0] + e : at[e], in = one ? (r < TS_PAGE_KEYS ? page[0] : page[1]) : page[e];
                    const bool good = (unsigned)in < (unsigned)num;
                    if (r >= 0 && !good) bits |= TS_STATUS_INDEX;
                    v[e] = r >= 0 && good ? in * TS_PAGE_KEYS + r % TS_PAGE_KEYS : -1;
                }
                if (a.slot_vec && i0 >= lo && i0 + 4 <= hi)
                    *reinterpret_cast<int4 *>(a.slot + i0) = make_int4(v[0], v[1], v[2], v[3]);
                else
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (i0 + e >= lo && i0 + e < hi) a.slot[i0 + e] = v[e];
            }
        }
        move();
        at.n += tile.n, at.take += tile.take, at.back += tile.back;
        if (base + kPageThreads < B) __syncthreads();   // shared memory is the next tile's
    }
    if (a.slot)
        for (long long i = max((long long)s0, at.n) + tid; i < s1; i += kPageThreads) a.slot[i] = -1;
    if (bits) flag(a.status, bits);

    // the last CTA to come here: every other one has read what is now written
    __syncthreads();
    if (ctas > 1) {
        if (tid == 0) {
            __threadfence();
            unsigned *done = (unsigned *)a.pool.ring_state + 2;
            last_s = atomicAdd(done, 1u) == ctas - 1;
            if (last_s) *done = 0;
            __threadfence();
        }
        __syncthreads();
        if (!last_s) return;
    }
    long long take = 0;
    for (int base = 0; base < B; base += kPageThreads) {
        const int b = base + tid;
        if (B > kPageThreads) {
            r = request(a, b);
            run = block_sums(r.own, part);
            ok = b < B && pool_ok && r.sound && (r.own.take == 0 || take + run.take <= count);
        }
        if (b < B) a.new_held[b] = ok ? (int)r.want : r.held;
        if (B > kPageThreads) {
            if (tid == kPageThreads - 1) tile_s = run;
            __syncthreads();
            take += tile_s.take;
        }
    }
    if (tid == 0) {
        a.new_state[0] = pool_ok ? ring_at(head + taken_s, num) : head;
        a.new_state[1] = pool_ok ? (int)(count - taken_s + all.back) : count;
    }
}

// --------------------------------------------------------------- rows by slot ----
// cache[slot / 64][h][slot % 64] = new[t][h]: 16-byte pieces, a CTA a token, the
// new row's loads under way before its slot is known. (Four tokens a CTA: 8 of 32
// heads 2.4 us for 1.4, 2048 of them 12.7 for 11.4, 16384 the same 80.6, which is
// 98 % of the copy rate.)
constexpr int kSlotThreads = 256;

__global__ void __launch_bounds__(kSlotThreads) k_append_slots(uint4 *k_pages, uint4 *v_pages, const uint4 *k_new,
                                                               const uint4 *v_new, long long k_stride,
                                                               long long v_stride, const int32_t *slot, int H,
                                                               int vec_log2, int num_pages, uint32_t *status) {
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x, per = H << vec_log2;
    for (int p = threadIdx.x; p < per; p += kSlotThreads) {
        const int at = slot[t];
        const uint4 k = __ldcs(k_new + t * k_stride + p), v = __ldcs(v_new + t * v_stride + p);
        const int page = at / TS_PAGE_KEYS, row = at % TS_PAGE_KEYS, h = p >> vec_log2, c = p & ((1 << vec_log2) - 1);
        if (at < 0 || page >= num_pages) {
            if (at != -1 && p == 0) flag(status, TS_STATUS_INDEX);
            continue;
        }
        const size_t dst = ((((size_t)page * H + h) * TS_PAGE_KEYS + row) << vec_log2) + c;
        k_pages[dst] = k;
        v_pages[dst] = v;
    }
}

}  // namespace

cudaError_t launch_pages_build(const ts_page_pool &pool, int32_t *new_held, int32_t *new_state, int32_t *slot,
                               int max_slots, int32_t *slot_offset, const int32_t *row_begin, const int32_t *row_end,
                               uint32_t *status, cudaStream_t s) {
    PageArgs a{pool, new_held, new_state, slot, slot_offset, row_begin, row_end, slot ? max_slots : 0, 0,
               ((uintptr_t)slot & 15) == 0, status};
    const int ctas = (int)std::min<long long>(2LL * num_sms(), 1 + (long long)a.max_slots / (8 * kPageThreads));
    a.per_cta = (int)(((long long)a.max_slots + ctas - 1) / ctas + 3) / 4 * 4;
    return launch(k_pages_build, dim3(ctas), dim3(kPageThreads), 0, s, a);
}

cudaError_t launch_append_slots(const ts_paged_kv &kv, const void *k_new, const void *v_new, long long k_stride,
                                long long v_stride, const int32_t *slot, int T, int H, int d, uint32_t *status,
                                cudaStream_t s) {
    return launch(k_append_slots, dim3(T), dim3(kSlotThreads), 0, s, (uint4 *)kv.k_pages, (uint4 *)kv.v_pages,
                  (const uint4 *)k_new, (const uint4 *)v_new, k_stride / 8, v_stride / 8, slot, H, d == 128 ? 4 : 3,
                  (int)kv.num_pages, status);
}

}  // namespace ts
