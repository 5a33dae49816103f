// Checks and argument structs that the C entry points of the attention side share. A cache
// is any of the ABI's cache structs: they agree in n_pages, kv_heads, page and head_dim.
#pragma once

#include "../../include/sparse_ffn_attention.h"
#include "attn_launch.hpp"
#include "status.hpp"

namespace sffn {

// Bounds that keep every size product below 2^63 and every grid below 2^31.
constexpr int64_t kMaxTokens = (int64_t)1 << 30;
// Of the cache: new tokens of a call and tokens of a sequence, so that every
// position, with a call's tokens added, fits 31 bits.
constexpr int64_t kMaxNewTokens = (int64_t)1 << 28;
constexpr int64_t kMaxCapacity = (int64_t)1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 42;
constexpr int64_t kMaxGrid = ((int64_t)1 << 31) - 1;
constexpr int32_t kMaxHeads = 65536;

inline size_t elem_size(int dtype) { return dtype == SFFN_BF16 ? 2 : 4; }

inline sffn_status_t check_dtype(int dtype) {
    if (dtype != SFFN_F32 && dtype != SFFN_BF16) return fail(SFFN_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    return SFFN_OK;
}

// A [T, heads, dim] view. wide: rows must be 16-byte aligned. out: elements
// must not overlap (tokens outside heads or heads outside tokens).
inline sffn_status_t check_heads(const sffn_heads_t* v, const char* name, int64_t T, int64_t heads, int64_t dim, int dtype,
                          bool wide, bool out) {
    if (!v || !v->data) return fail(SFFN_ERR_INVALID_ARG, "%s is null", name);
    if (v->stride_token < 0 || v->stride_head < 0 || v->stride_token > kMaxStride || v->stride_head > kMaxStride)
        return fail(SFFN_ERR_INVALID_ARG, "%s has strides out of range (%lld, %lld)", name,
                    (long long)v->stride_token, (long long)v->stride_head);
    int64_t a, b, last;
    if (__builtin_mul_overflow(T - 1, v->stride_token, &a) || __builtin_mul_overflow(heads - 1, v->stride_head, &b) ||
        __builtin_add_overflow(a, b, &last) || last > ((int64_t)1 << 60))
        return fail(SFFN_ERR_INVALID_ARG, "%s is too large", name);
    const size_t e = elem_size(dtype);
    if (reinterpret_cast<uintptr_t>(v->data) % e != 0)
        return fail(SFFN_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
    if (wide && (!aligned16(v->data) || (size_t)v->stride_token * e % 16 != 0 || (size_t)v->stride_head * e % 16 != 0))
        return fail(SFFN_ERR_INVALID_ARG, "%s must have 16-byte aligned rows", name);
    if (out) {
        const bool heads_inside = (heads == 1 || v->stride_head >= dim) && (T == 1 || v->stride_token >= b + dim);
        const bool tokens_inside = (T == 1 || v->stride_token >= dim) && (heads == 1 || v->stride_head >= a + dim);
        if (!heads_inside && !tokens_inside) return fail(SFFN_ERR_INVALID_ARG, "%s overlaps itself", name);
    }
    return SFFN_OK;
}

inline Heads view(const sffn_heads_t* v) {
    return v ? Heads{v->data, v->stride_token, v->stride_head} : Heads{nullptr, 0, 0};
}

#define SFFN_TRY(call)                            \
    do {                                          \
        const sffn_status_t try_st = (call);      \
        if (try_st != SFFN_OK) return try_st;     \
    } while (0)

// ---- cache ---------------------------------------------------------------------------

template <typename Cache>
sffn_status_t check_cache(const Cache* c, const sffn_kv_batch_t* b, int64_t T) {
    if (!c || !b) return fail(SFFN_ERR_INVALID_ARG, "cache and batch must not be null");
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
        return fail(SFFN_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128 (got %d)", c->page);
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(SFFN_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 (got %d)", c->head_dim);
    if (c->kv_heads < 1 || c->kv_heads > kMaxHeads)
        return fail(SFFN_ERR_INVALID_ARG, "kv_heads must be positive (got %d)", c->kv_heads);
    if (c->n_pages < 1 || c->n_pages > INT32_MAX)
        return fail(SFFN_ERR_INVALID_ARG, "n_pages must lie in [1, 2^31) (got %lld)", (long long)c->n_pages);
    if (b->n_seqs < 0 || b->max_pages < 0 || b->max_new < 0 || b->max_kv < 0)
        return fail(SFFN_ERR_INVALID_ARG, "n_seqs, max_pages, max_new and max_kv must not be negative");
    if (b->table_stride < 0 || b->table_stride > kMaxStride || (b->n_seqs > 1 && b->table_stride < b->max_pages))
        return fail(SFFN_ERR_INVALID_ARG, "table_stride %lld does not fit rows of %d pages",
                    (long long)b->table_stride, b->max_pages);
    if (T < 0) return fail(SFFN_ERR_INVALID_ARG, "T must be >= 0 (got %lld)", (long long)T);
    if (T > kMaxNewTokens) return fail(SFFN_ERR_UNSUPPORTED, "T = %lld is too large for one call", (long long)T);
    if ((int64_t)b->max_pages * c->page > kMaxCapacity)
        return fail(SFFN_ERR_UNSUPPORTED, "max_pages %d of %d tokens are too many", b->max_pages, c->page);
    if (!b->cu && T != b->n_seqs)
        return fail(SFFN_ERR_INVALID_ARG, "without cu, T must be n_seqs (got %lld, %d)", (long long)T, b->n_seqs);
    if (!b->cu && T > 0 && b->max_new < 1)
        return fail(SFFN_ERR_INVALID_ARG, "max_new must be positive (got %d)", b->max_new);
    return SFFN_OK;
}

// The four buffers of a cache and their names.
struct CacheBuffers {
    const void* p[4];
    const char* name[4];
};

inline sffn_status_t check_cache_pointers(const CacheBuffers& c, const sffn_kv_batch_t* b) {
    for (int i = 0; i < 4; ++i) {
        if (!c.p[i]) return fail(SFFN_ERR_INVALID_ARG, "%s is null", c.name[i]);
        if (!aligned16(c.p[i])) return fail(SFFN_ERR_INVALID_ARG, "%s is not 16-byte aligned", c.name[i]);
    }
    if (b->max_pages < 1) return fail(SFFN_ERR_INVALID_ARG, "max_pages must be positive (got %d)", b->max_pages);
    if (!b->kv_lens || !b->block_table)
        return fail(SFFN_ERR_INVALID_ARG, "block_table and kv_lens must not be null");
    for (const void* p : {(const void*)b->block_table, (const void*)b->kv_lens, (const void*)b->cu})
        if (reinterpret_cast<uintptr_t>(p) % 4 != 0)
            return fail(SFFN_ERR_INVALID_ARG, "block_table, kv_lens and cu must be 4-byte aligned");
    return SFFN_OK;
}

// Everything but the buffers.
template <typename Cache>
CacheArgs cache_shape(const Cache* c, const sffn_kv_batch_t* b, int dtype, int64_t T) {
    CacheArgs a{};
    a.n_pages = c->n_pages;
    a.Hkv = c->kv_heads;
    a.P = c->page;
    a.D = c->head_dim;
    a.shift = __builtin_ctz((unsigned)c->page);
    a.table = b->block_table;
    a.table_stride = b->table_stride;
    a.lens = b->kv_lens;
    a.cu = b->cu;
    a.B = b->n_seqs;
    a.max_pages = b->max_pages;
    // no sequence has more new tokens than the call, and without offsets each has one
    a.max_new = !b->cu ? 1 : (int)(b->max_new < T ? b->max_new : T);
    a.max_kv = b->max_kv;
    a.T = T;
    a.dt = dtype == SFFN_BF16 ? Dt::BF16 : Dt::F32;
    return a;
}

// The checks of attention that its workspace size needs too.
template <typename Cache>
sffn_status_t check_attention(const Cache* cache, const sffn_kv_batch_t* batch, int32_t n_q_heads,
                              int32_t window, int64_t T) {
    SFFN_TRY(check_cache(cache, batch, T));
    if (n_q_heads < 1 || n_q_heads > kMaxHeads || n_q_heads % cache->kv_heads != 0)
        return fail(SFFN_ERR_INVALID_ARG, "n_q_heads must be a multiple of kv_heads (got %d, %d)", n_q_heads,
                    cache->kv_heads);
    if (window < 0) return fail(SFFN_ERR_INVALID_ARG, "window must be >= 0 (got %d)", window);
    if (T * n_q_heads > kMaxGrid)
        return fail(SFFN_ERR_UNSUPPORTED, "T = %lld is too large for one call", (long long)T);
    return SFFN_OK;
}

inline sffn_status_t make_plan(const CacheArgs& a, int32_t n_q_heads, int32_t window,
                               AttnPlan (*plan_of)(const CacheArgs&, int, int), AttnPlan* plan,
                               int unit_cost = 0) {
    const int64_t tiles = ((int64_t)a.max_new * (n_q_heads / a.Hkv) + 15) / 16;
    if (tiles > kMaxGrid || (int64_t)a.B * a.Hkv > kMaxGrid / (tiles > 0 ? tiles : 1))
        return fail(SFFN_ERR_UNSUPPORTED, "the batch is too large for one call");
    // the kernels' counts of steps of 64 keys over all sequences and heads
    const int64_t steps = (int64_t)a.max_pages * a.P / 64 + 8 + unit_cost;
    if ((int64_t)a.B * a.Hkv > kMaxGrid / steps)
        return fail(SFFN_ERR_UNSUPPORTED, "%d sequences of %d pages are too many for one call", a.B, a.max_pages);
    *plan = plan_of(a, n_q_heads, window);
    if (plan->blocks > kMaxGrid) return fail(SFFN_ERR_UNSUPPORTED, "the batch is too large for one call");
    return SFFN_OK;
}

// The workspace that a plan needs.
inline sffn_status_t check_workspace(const void* workspace, size_t ws_bytes, size_t need) {
    if (need == 0) return SFFN_OK;
    if (!workspace) return fail(SFFN_ERR_INVALID_ARG, "workspace is null");
    if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
        return fail(SFFN_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
    if (ws_bytes < need) return fail(SFFN_ERR_WORKSPACE, "workspace holds %zu bytes, %zu needed", ws_bytes, need);
    return SFFN_OK;
}

}  // namespace sffn
