// api_decode.cu -- C ABI of a decode step on the paged cache: argument checks
// and dispatch. Declared, with meaning, layouts and error behaviour, in
// include/treespec.h.
#include <math.h>

#include "decode.cuh"

namespace {

using ts::set_error;

ts_status done(cudaError_t e, const char *who) {
    if (e != cudaSuccess) return set_error(TS_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return set_error(TS_OK, "%s", "");
}

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Arrays of 32-bit numbers; a NULL one is as good as aligned.
template <typename... P>
ts_status check_words(const char *who, P... p) {
    if ((... && aligned(p, 4))) return TS_OK;
    return set_error(TS_ERR_INVALID_ARG, "%s: an array of 32-bit numbers is not 4-byte aligned", who);
}

// Whether two arrays of so many 32-bit numbers share any (NULL: none).
bool overlap(const void *p, long long n, const void *q, long long m) {
    return p && q && (uintptr_t)p < (uintptr_t)q + 4 * m && (uintptr_t)q < (uintptr_t)p + 4 * n;
}

ts_status check_pages(const ts_paged_kv *kv, int H, int d, const char *who) {
    if (!kv) return set_error(TS_ERR_INVALID_ARG, "%s: cache is NULL", who);
    if (!kv->k_pages || !kv->v_pages) return set_error(TS_ERR_INVALID_ARG, "%s: pages are NULL", who);
    if (!aligned(kv->k_pages, 16) || !aligned(kv->v_pages, 16))
        return set_error(TS_ERR_INVALID_ARG, "%s: pages must be 16-byte aligned", who);
    if (d != 64 && d != 128) return set_error(TS_ERR_UNSUPPORTED, "%s: head_dim %d (supported: 64, 128)", who, d);
    if (H < 1 || H > 65535) return set_error(TS_ERR_INVALID_ARG, "%s: H=%d outside [1, 65535]", who, H);
    if (kv->num_pages < 1) return set_error(TS_ERR_INVALID_ARG, "%s: num_pages=%d", who, kv->num_pages);
    return TS_OK;
}

ts_status check_stride(const void *p, long long row, long long stride, const char *what, const char *who) {
    if (!p) return set_error(TS_ERR_INVALID_ARG, "%s: %s is NULL", who, what);
    if (!aligned(p, 16)) return set_error(TS_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", who, what);
    if (stride < row || stride % 8 != 0 || stride > (1LL << 31))
        return set_error(TS_ERR_INVALID_ARG, "%s: %s stride %lld (at least H * d = %lld, a multiple of 16 bytes)", who,
                         what, stride, row);
    return TS_OK;
}

bool decode_sizes_ok(int B, int Hq, int Hkv, int d) {
    return B >= 1 && B <= 65535 && Hkv >= 1 && Hkv <= 65535 && Hq >= 1 && Hq <= 65535 && Hq % Hkv == 0 &&
           (d == 64 || d == 128) && (long long)B * Hq < (1LL << 31);
}

}  // namespace

extern "C" {

ts_status kv_pages_build(const ts_page_pool *pool, int32_t *new_held, int32_t *new_state, int32_t *slot,
                         int max_slots, int32_t *slot_offset, const int32_t *row_begin, const int32_t *row_end,
                         uint32_t *status, cudaStream_t stream) {
    const char *who = "kv_pages_build";
    if (!pool) return set_error(TS_ERR_INVALID_ARG, "%s: pool is NULL", who);
    if (!pool->block_table || !pool->held || !pool->ring || !pool->ring_state || !new_held || !new_state || !row_end)
        return set_error(TS_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (pool->B < 1 || pool->B > 65535) return set_error(TS_ERR_INVALID_ARG, "%s: B=%d outside [1, 65535]", who, pool->B);
    if (pool->max_pages < 1 || pool->max_pages > (1 << 24) || pool->num_pages < 1 || pool->num_pages >= (1 << 25))
        return set_error(TS_ERR_INVALID_ARG, "%s: num_pages=%d, max_pages=%d", who, pool->num_pages, pool->max_pages);
    if (slot && (max_slots < 1 || !row_begin))
        return set_error(TS_ERR_INVALID_ARG, "%s: slots need row_begin and max_slots >= 1 (%d)", who, max_slots);
    if (slot_offset && !slot) return set_error(TS_ERR_INVALID_ARG, "%s: slot_offset without slots", who);
    const ts_status st = check_words(who, pool->block_table, pool->held, pool->ring, pool->ring_state, new_held, new_state,
                                     slot, slot_offset, row_begin, row_end, status);
    if (st) return st;
    return done(ts::launch_pages_build(*pool, new_held, new_state, slot, slot ? max_slots : 0, slot_offset,
                                       slot ? row_begin : nullptr, row_end, status, stream),
                who);
}

ts_status kv_append_slots(const ts_paged_kv *kv, const void *k_new, const void *v_new, long long k_stride,
                          long long v_stride, const int32_t *slot, int T, int H, int d, uint32_t *status,
                          cudaStream_t stream) {
    const char *who = "kv_append_slots";
    ts_status st = check_pages(kv, H, d, who);
    if (st) return st;
    if (kv->num_pages >= (1 << 25)) return set_error(TS_ERR_INVALID_ARG, "%s: num_pages=%d", who, kv->num_pages);
    if (T < 1) return set_error(TS_ERR_INVALID_ARG, "%s: T=%d must be >= 1", who, T);
    if (!slot) return set_error(TS_ERR_INVALID_ARG, "%s: slot is NULL", who);
    if ((st = check_stride(k_new, (long long)H * d, k_stride, "k_new", who)) ||
        (st = check_stride(v_new, (long long)H * d, v_stride, "v_new", who)) || (st = check_words(who, slot, status)))
        return st;
    return done(ts::launch_append_slots(*kv, k_new, v_new, k_stride, v_stride, slot, T, H, d, status, stream), who);
}

ts_status decode_attention_paged(void *out, const void *q, long long q_stride, const ts_paged_kv *kv,
                                 const int32_t *kv_len, int B, int Hq, int Hkv, int d, float scale, void *ws,
                                 size_t ws_bytes, uint32_t *status, cudaStream_t stream) {
    const char *who = "decode_attention_paged";
    ts_status st = check_pages(kv, Hkv, d, who);
    if (st) return st;
    if (!kv->block_table || kv->max_pages < 1 || kv->max_pages > (1 << 24))
        return set_error(TS_ERR_INVALID_ARG, "%s: block table of %d pages a request", who, kv->max_pages);
    if (!out || !kv_len) return set_error(TS_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned(out, 16)) return set_error(TS_ERR_INVALID_ARG, "%s: out must be 16-byte aligned", who);
    if (!decode_sizes_ok(B, Hq, Hkv, d))
        return set_error(TS_ERR_INVALID_ARG, "%s: B=%d, Hq=%d (a multiple of Hkv=%d), B * Hq below 2^31", who, B, Hq, Hkv);
    if ((st = check_stride(q, (long long)Hq * d, q_stride, "q", who)) ||
        (st = check_words(who, kv_len, kv->block_table, status)))
        return st;
    if (out == q) return set_error(TS_ERR_INVALID_ARG, "%s: out needs a place of its own", who);
    if (!(scale > 0.f)) scale = 1.0f / sqrtf((float)d);
    if (!(scale * 1.4426950408889634f < INFINITY))   // scores are exponents of 2
        return set_error(TS_ERR_INVALID_ARG, "%s: scale is not finite, or its product with log2(e) is not", who);
    const size_t need = ts::decode_ws_bytes(B, Hq, Hkv, d);
    if (!ws || ws_bytes < need)
        return set_error(TS_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", who, need,
                         ws ? ws_bytes : (size_t)0);
    if (!aligned(ws, 16)) return set_error(TS_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", who);
    return done(ts::launch_attn_decode(out, q, q_stride, *kv, kv_len, B, Hq, Hkv, d, scale, ws, status, stream), who);
}

size_t treespec_decode_workspace_size(int B, int Hq, int Hkv, int d) {
    return decode_sizes_ok(B, Hq, Hkv, d) ? ts::decode_ws_bytes(B, Hq, Hkv, d) : 0;
}

ts_status sample_tokens(int32_t *token, float *probs, float *kept, const void *logits, long long row_stride,
                        ts_dtype dtype, const float *u, const float *temperature, const int32_t *top_k,
                        const float *top_p, const float *min_p, int R, int V, uint32_t *status, cudaStream_t stream) {
    const char *who = "sample_tokens";
    if (dtype != TS_F32 && dtype != TS_BF16) return set_error(TS_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dtype);
    if (!logits) return set_error(TS_ERR_INVALID_ARG, "%s: logits is NULL", who);
    if (!aligned(logits, dtype == TS_BF16 ? 2 : 4))
        return set_error(TS_ERR_INVALID_ARG, "%s: logits must be aligned to their type", who);
    if (R < 1) return set_error(TS_ERR_INVALID_ARG, "%s: R=%d must be >= 1", who, R);
    if (V < 1 || V > (1 << 18)) return set_error(TS_ERR_INVALID_ARG, "%s: V=%d outside [1, 2^18]", who, V);
    if (row_stride < V || row_stride > (1LL << 31))
        return set_error(TS_ERR_INVALID_ARG, "%s: row stride %lld below V=%d or above 2^31", who, row_stride, V);
    if (!token && !probs && !kept) return set_error(TS_ERR_INVALID_ARG, "%s: no output is asked for", who);
    if (token && !u) return set_error(TS_ERR_INVALID_ARG, "%s: a token needs u", who);
    if ((const void *)probs == logits || (probs && probs == kept))
        return set_error(TS_ERR_INVALID_ARG, "%s: probs needs a place of its own", who);
    if ((const void *)kept == logits && (dtype != TS_F32 || row_stride != V))
        return set_error(TS_ERR_INVALID_ARG, "%s: kept in the logits' place only where these are fp32, V apart", who);
    if (token && (const void *)token == logits)
        return set_error(TS_ERR_INVALID_ARG, "%s: token needs a place of its own", who);
    const ts_status st = check_words(who, token, probs, kept, u, temperature, top_k, top_p, min_p, status);
    if (st) return st;
    // a row's CTAs read other rows' settings too, whose CTAs may already write
    const void *const set[] = {u, temperature, top_k, top_p, min_p};
    for (const void *p : set) {
        const char *const what = overlap(token, R, p, R)                    ? "token"
                                 : overlap(probs, (long long)R * V, p, R) ? "probs"
                                 : overlap(kept, (long long)R * V, p, R)  ? "kept"
                                                                          : nullptr;
        if (what)
            return set_error(TS_ERR_INVALID_ARG, "%s: %s needs a place of its own, apart from u and the settings", who, what);
    }
    const ts::SampleArgs a{token, probs, kept,  logits, row_stride, u, temperature,
                           top_k, top_p, min_p, R,      V,          status};
    return done(ts::launch_sample(a, dtype, stream), who);
}

}  // extern "C"
