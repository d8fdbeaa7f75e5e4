// api_kv8.cu -- C ABI of the 8-bit KV cache and of the head norms with
// rotation: argument checks and dispatch. Declared, with meaning, layouts and
// error behaviour, in include/treespec.h.
#include <math.h>

#include "kv8.cuh"

namespace {

using ts::set_error;

ts_status done(cudaError_t e, const char *who) {
    if (e != cudaSuccess) return set_error(TS_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return set_error(TS_OK, "%s", "");
}

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

ts_status check_tree8(const ts_tree *t, const char *who) {
    if (!t) return set_error(TS_ERR_INVALID_ARG, "%s: tree is NULL", who);
    if (t->B < 1 || t->B > 65535) return set_error(TS_ERR_INVALID_ARG, "%s: tree B=%d outside [1, 65535]", who, t->B);
    if (t->n_max < 1 || t->n_max > TS_MAX_NODES)
        return set_error(TS_ERR_INVALID_ARG, "%s: tree n_max=%d outside [1, %d]", who, t->n_max, TS_MAX_NODES);
    if (!t->n_nodes || !t->perm || !t->dfs_of || !t->sub_end)
        return set_error(TS_ERR_INVALID_ARG, "%s: a tree array is NULL", who);
    return TS_OK;
}

ts_status check_dim(int d, const char *who) {
    if (d != 64 && d != 128) return set_error(TS_ERR_UNSUPPORTED, "%s: head_dim %d (supported: 64, 128)", who, d);
    return TS_OK;
}

ts_status check_kv8(const ts_kv8 *kv, const char *who) {
    if (!kv) return set_error(TS_ERR_INVALID_ARG, "%s: cache is NULL", who);
    if (!kv->k || !kv->v || !kv->k_scale || !kv->v_scale)
        return set_error(TS_ERR_INVALID_ARG, "%s: a cache array is NULL", who);
    ts_status st = check_dim(kv->d, who);
    if (st) return st;
    if (kv->B < 1 || kv->B > 65535 || kv->H < 1 || kv->H > 65535)
        return set_error(TS_ERR_INVALID_ARG, "%s: cache B=%d, H=%d outside [1, 65535]", who, kv->B, kv->H);
    long long rows;
    if (kv->block_table) {
        if (kv->num_pages < 1 || kv->max_pages < 1 || kv->max_pages > (1 << 24))
            return set_error(TS_ERR_INVALID_ARG, "%s: num_pages=%d, max_pages=%d", who, kv->num_pages, kv->max_pages);
        rows = (long long)kv->num_pages * kv->H * TS_PAGE_KEYS;
    } else {
        if (kv->L_max < 1) return set_error(TS_ERR_INVALID_ARG, "%s: L_max=%d must be >= 1", who, kv->L_max);
        rows = (long long)kv->B * kv->H * kv->L_max;
    }
    if (rows >= (1LL << 31) - 256)
        return set_error(TS_ERR_INVALID_ARG, "%s: %lld cache rows (2^31 - 256 or more)", who, rows);
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16))
        return set_error(TS_ERR_INVALID_ARG, "%s: codes must be 16-byte aligned", who);
    if (!aligned(kv->k_scale, 4) || !aligned(kv->v_scale, 4))
        return set_error(TS_ERR_INVALID_ARG, "%s: scales must be 4-byte aligned", who);
    return TS_OK;
}

ts_status check_kv8_tree(const ts_kv8 *kv, const ts_tree *t, const char *who) {
    ts_status st = check_tree8(t, who);
    if (st || (st = check_kv8(kv, who))) return st;
    if (kv->B != t->B) return set_error(TS_ERR_INVALID_ARG, "%s: cache B=%d, tree B=%d", who, kv->B, t->B);
    if (ts::kv8_rows(*kv) < t->n_max)
        return set_error(TS_ERR_INVALID_ARG, "%s: %d cache rows below n_max=%d", who, ts::kv8_rows(*kv), t->n_max);
    return TS_OK;
}

// One projection's node rows: H heads of d, `stride` elements apart.
ts_status check_rows(const void *p, int H, int d, long long stride, ts_dtype dt, const char *what, const char *who) {
    const int es = dt == TS_BF16 ? 2 : 4;
    if (!p) return set_error(TS_ERR_INVALID_ARG, "%s: %s is NULL", who, what);
    if (!aligned(p, 16)) return set_error(TS_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned", who, what);
    if (stride < (long long)H * d || stride * es % 16 != 0 || stride > (1LL << 31))
        return set_error(TS_ERR_INVALID_ARG, "%s: %s stride %lld (at least H * d = %lld, a multiple of 16 bytes)", who,
                         what, stride, (long long)H * d);
    return TS_OK;
}

ts_status check_dtype(ts_dtype dt, const char *who) {
    if (dt != TS_F32 && dt != TS_BF16) return set_error(TS_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dt);
    return TS_OK;
}

ts_status check_rope(const ts_qk_rope *r, const ts_tree *t, int d, const char *who) {
    if (r->rot_dim < 0 || r->rot_dim > d || r->rot_dim % 16 != 0)
        return set_error(TS_ERR_UNSUPPORTED, "%s: rot_dim %d (a multiple of 16 up to head_dim %d)", who, r->rot_dim, d);
    if (r->rot_dim && !r->inv_freq) return set_error(TS_ERR_INVALID_ARG, "%s: inv_freq is NULL", who);
    if (r->rot_dim && !t->pos)
        return set_error(TS_ERR_INVALID_ARG, "%s: the tree has no positions (tree_build with prefix_len)", who);
    if (r->norm && !(r->eps >= 0.f)) return set_error(TS_ERR_INVALID_ARG, "%s: eps must be >= 0", who);
    return TS_OK;
}

}  // namespace

extern "C" {

ts_status tree_qk_norm_rope(void *q_out, void *k_out, const void *q, const void *k, int Hq, int Hk, int d,
                            long long q_stride, long long k_stride, const ts_qk_rope *rope, const ts_tree *t,
                            ts_dtype dtype, uint32_t *status, cudaStream_t stream) {
    const char *who = "tree_qk_norm_rope";
    (void)status;
    ts_status st = check_tree8(t, who);
    if (st || (st = check_dim(d, who)) || (st = check_dtype(dtype, who))) return st;
    if (!rope) return set_error(TS_ERR_INVALID_ARG, "%s: rope is NULL", who);
    if ((st = check_rope(rope, t, d, who))) return st;
    if (Hq < 0 || Hk < 0 || Hq + Hk < 1 || Hq > 65535 || Hk > 65535)
        return set_error(TS_ERR_INVALID_ARG, "%s: Hq=%d, Hk=%d", who, Hq, Hk);
    if (Hq && ((st = check_rows(q, Hq, d, q_stride, dtype, "q", who)) ||
               (st = check_rows(q_out, Hq, d, (long long)Hq * d, dtype, "q_out", who))))
        return st;
    if (Hk && ((st = check_rows(k, Hk, d, k_stride, dtype, "k", who)) ||
               (st = check_rows(k_out, Hk, d, (long long)Hk * d, dtype, "k_out", who))))
        return st;
    if ((Hq && q_out == q && q_stride != (long long)Hq * d) || (Hk && k_out == k && k_stride != (long long)Hk * d))
        return set_error(TS_ERR_INVALID_ARG, "%s: in place only on contiguous heads", who);
    return done(ts::launch_qk_norm_rope(q_out, k_out, q, k, Hq, Hk, d, q_stride, k_stride, *rope, *t, dtype, stream), who);
}

ts_status kv8_append(const ts_kv8 *kv, const void *k_new, const void *v_new, long long k_stride, long long v_stride,
                     const ts_qk_rope *rope, void *q_out, const void *q, int Hq, long long q_stride,
                     const int32_t *prefix_len, const ts_tree *t, ts_dtype dtype, uint32_t *status,
                     cudaStream_t stream) {
    const char *who = "kv8_append";
    ts_status st = check_kv8_tree(kv, t, who);
    if (st || (st = check_dtype(dtype, who))) return st;
    if (!prefix_len) return set_error(TS_ERR_INVALID_ARG, "%s: prefix_len is NULL", who);
    if ((st = check_rows(k_new, kv->H, kv->d, k_stride, dtype, "k_new", who)) ||
        (st = check_rows(v_new, kv->H, kv->d, v_stride, dtype, "v_new", who)))
        return st;
    if (rope && (st = check_rope(rope, t, kv->d, who))) return st;
    if (Hq < 0 || Hq > 65535 || (Hq && !rope))
        return set_error(TS_ERR_INVALID_ARG, "%s: Hq=%d%s", who, Hq, Hq > 0 && !rope ? " without rope" : "");
    if (Hq && ((st = check_rows(q, Hq, kv->d, q_stride, dtype, "q", who)) ||
               (st = check_rows(q_out, Hq, kv->d, (long long)Hq * kv->d, dtype, "q_out", who))))
        return st;
    if (Hq && q_out == q && q_stride != (long long)Hq * kv->d)
        return set_error(TS_ERR_INVALID_ARG, "%s: in place only on contiguous heads", who);
    return done(ts::launch_kv8_append(*kv, k_new, v_new, k_stride, v_stride, rope, q_out, q, Hq, q_stride, prefix_len,
                                      *t, dtype, status, stream),
                who);
}

ts_status kv8_read(void *k_out, void *v_out, const ts_kv8 *kv, const int32_t *row_begin, const int32_t *row_end,
                   int L_out, ts_dtype dtype, uint32_t *status, cudaStream_t stream) {
    const char *who = "kv8_read";
    ts_status st = check_kv8(kv, who);
    if (st || (st = check_dtype(dtype, who))) return st;
    if (!k_out || !v_out || !row_end) return set_error(TS_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned(k_out, 16) || !aligned(v_out, 16))
        return set_error(TS_ERR_INVALID_ARG, "%s: outputs must be 16-byte aligned", who);
    if (L_out < 1) return set_error(TS_ERR_INVALID_ARG, "%s: L_out=%d must be >= 1", who, L_out);
    return done(ts::launch_kv8_read(k_out, v_out, *kv, row_begin, row_end, L_out, dtype, status, stream), who);
}

ts_status tree_attention_kv8(void *out, const void *q, const ts_kv8 *kv, int Hq, const int32_t *prefix_len,
                             const ts_tree *t, float scale, void *ws, size_t ws_bytes, uint32_t *status,
                             cudaStream_t stream) {
    const char *who = "tree_attention_kv8";
    ts_status st = check_kv8_tree(kv, t, who);
    if (st) return st;
    if (!out || !q || !prefix_len) return set_error(TS_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned(out, 16) || !aligned(q, 16))
        return set_error(TS_ERR_INVALID_ARG, "%s: q and out must be 16-byte aligned", who);
    if (Hq < 1 || Hq > 65535 || Hq % kv->H != 0)
        return set_error(TS_ERR_INVALID_ARG, "%s: Hq=%d is not a multiple of the cache's H=%d", who, Hq, kv->H);
    if ((long long)t->B * Hq * t->n_max >= (1LL << 31))
        return set_error(TS_ERR_INVALID_ARG, "%s: %lld query rows (2^31 or more)", who, (long long)t->B * Hq * t->n_max);
    if (!(scale > 0.f)) scale = 1.0f / sqrtf((float)kv->d);
    if (!(scale * ts::kLog2e < INFINITY))   // the kernel's scores are exponents of 2
        return set_error(TS_ERR_INVALID_ARG, "%s: scale is not finite, or its product with log2(e) is not", who);
    const size_t need = ts::kv8_attention_ws_bytes(t->B, Hq, kv->H, t->n_max, kv->d, ts::kv8_rows(*kv));
    if (!ws || ws_bytes < need)
        return set_error(TS_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", who, need,
                         ws ? ws_bytes : (size_t)0);
    if (!aligned(ws, 16)) return set_error(TS_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", who);
    const char *why = nullptr;
    const cudaError_t e = ts::launch_attn_kv8(out, q, *kv, Hq, prefix_len, *t, scale, ws, status, stream, &why);
    if (why) return set_error(TS_ERR_CUDA, "%s: %s", who, why);
    return done(e, who);
}

ts_status kv8_commit(const ts_kv8 *kv, const int32_t *prefix_len, int32_t *new_prefix_len, const int32_t *out_path,
                     const int32_t *out_count, const ts_tree *t, uint32_t *status, cudaStream_t stream) {
    const char *who = "kv8_commit";
    ts_status st = check_kv8_tree(kv, t, who);
    if (st) return st;
    if (!prefix_len || !new_prefix_len || !out_path || !out_count)
        return set_error(TS_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (new_prefix_len == prefix_len)
        return set_error(TS_ERR_INVALID_ARG, "%s: new_prefix_len aliases prefix_len", who);
    return done(ts::launch_kv8_commit(*kv, prefix_len, new_prefix_len, out_path, out_count, *t, status, stream), who);
}

size_t treespec_kv8_workspace_size(int B, int Hq, int Hkv, int n_max, int d, int L_max) {
    if (B < 1 || B > 65535 || Hkv < 1 || Hkv > 65535 || Hq < 1 || Hq > 65535 || Hq % Hkv != 0 || n_max < 1 ||
        n_max > TS_MAX_NODES || (d != 64 && d != 128) || L_max < n_max || (long long)B * Hq * n_max >= (1LL << 31))
        return 0;
    return ts::kv8_attention_ws_bytes(B, Hq, Hkv, n_max, d, L_max);
}

}  // extern "C"
