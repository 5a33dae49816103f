// C ABI of the attention-side operators (include/sparse_ffn_attention.h):
// argument checks, workspace sizes and the calls of the launchers.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/sparse_ffn_attention.h"
#include "attn_launch.hpp"
#include "status.hpp"

namespace {

using sffn::aligned16;
using sffn::as_int;
using sffn::fail;
using sffn::hip_status;

// Bounds that keep every size product below 2^63 and every grid below 2^31.
constexpr int64_t kMaxTokens = (int64_t)1 << 30;
// Of the cache: new tokens of a call and tokens of a sequence, so that every
// position, with a call's tokens added, fits 31 bits.
constexpr int64_t kMaxNewTokens = (int64_t)1 << 28;
constexpr int64_t kMaxCapacity = (int64_t)1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 42;
constexpr int64_t kMaxGrid = ((int64_t)1 << 31) - 1;
constexpr int32_t kMaxHeads = 65536;

size_t elem_size(int dtype) { return dtype == SFFN_BF16 ? 2 : 4; }

sffn_status_t check_dtype(int dtype) {
    if (dtype != SFFN_F32 && dtype != SFFN_BF16) return fail(SFFN_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    return SFFN_OK;
}

// A [T, heads, dim] view. wide: rows must be 16-byte aligned. out: elements
// must not overlap (tokens outside heads or heads outside tokens).
sffn_status_t check_heads(const sffn_heads_t* v, const char* name, int64_t T, int64_t heads, int64_t dim, int dtype,
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

sffn::Heads view(const sffn_heads_t* v) {
    return v ? sffn::Heads{v->data, v->stride_token, v->stride_head} : sffn::Heads{nullptr, 0, 0};
}

#define SFFN_TRY(call)                            \
    do {                                          \
        const sffn_status_t try_st = (call);      \
        if (try_st != SFFN_OK) return try_st;     \
    } while (0)

// ---- head norms and rotary positions -------------------------------------------

sffn_status_t check_rope(const sffn_rope_config_t* c) {
    if (!c) return fail(SFFN_ERR_INVALID_ARG, "config is null");
    if (c->n_q_heads < 1 || c->n_k_heads < 0 || c->n_q_heads > kMaxHeads || c->n_k_heads > kMaxHeads)
        return fail(SFFN_ERR_INVALID_ARG, "n_q_heads must be positive, n_k_heads not negative (got %d, %d)",
                    c->n_q_heads, c->n_k_heads);
    if (c->head_dim < 1 || c->head_dim > 512)
        return fail(SFFN_ERR_INVALID_ARG, "head_dim must lie in [1, 512] (got %d)", c->head_dim);
    if (c->rot_dim < 0 || c->rot_dim > c->head_dim || c->rot_dim % 2 != 0)
        return fail(SFFN_ERR_INVALID_ARG, "rot_dim must be even and lie in [0, head_dim] (got %d)", c->rot_dim);
    if (c->rot_dim > 0 && c->max_pos < 1)
        return fail(SFFN_ERR_INVALID_ARG, "max_pos must be positive (got %d)", c->max_pos);
    SFFN_TRY(check_dtype(as_int(c->dtype)));
    const int layout = as_int(c->layout);
    if (layout != SFFN_ROPE_HALF && layout != SFFN_ROPE_INTERLEAVED)
        return fail(SFFN_ERR_INVALID_ARG, "unknown layout %d", layout);
    if (c->norm != 0 && c->norm != 1) return fail(SFFN_ERR_INVALID_ARG, "norm must be 0 or 1 (got %d)", c->norm);
    if (c->norm && !(c->eps > 0.f && std::isfinite(c->eps)))
        return fail(SFFN_ERR_INVALID_ARG, "eps must be positive and finite (got %g)", (double)c->eps);
    return SFFN_OK;
}

// What forward and backward check alike: the token count, the table and weights.
sffn_status_t check_rope_inputs(const sffn_rope_config_t* c, const int32_t* positions, const float* table,
                                const void* q_weight, const void* k_weight, int64_t T) {
    if (T > kMaxTokens || T * (c->n_q_heads + c->n_k_heads) > kMaxGrid)
        return fail(SFFN_ERR_UNSUPPORTED, "T = %lld is too large for one call", (long long)T);
    if (c->rot_dim > 0 && (!positions || !table))
        return fail(SFFN_ERR_INVALID_ARG, "positions and table must not be null");
    if (reinterpret_cast<uintptr_t>(positions) % 4 != 0 || reinterpret_cast<uintptr_t>(table) % 4 != 0)
        return fail(SFFN_ERR_INVALID_ARG, "positions and table must be 4-byte aligned");
    const size_t e = elem_size(as_int(c->dtype));
    if (reinterpret_cast<uintptr_t>(q_weight) % e != 0 || reinterpret_cast<uintptr_t>(k_weight) % e != 0)
        return fail(SFFN_ERR_INVALID_ARG, "the weights are not aligned to their elements");
    return SFFN_OK;
}

sffn::RopeArgs rope_args(const sffn_rope_config_t* c, const int32_t* positions, const float* table,
                         const void* q_weight, const void* k_weight, int64_t T) {
    sffn::RopeArgs a{};
    a.dt = as_int(c->dtype) == SFFN_BF16 ? sffn::Dt::BF16 : sffn::Dt::F32;
    a.n_q = c->n_q_heads;
    a.n_k = c->n_k_heads;
    a.D = c->head_dim;
    a.R = c->rot_dim;
    a.max_pos = c->max_pos;
    a.interleaved = as_int(c->layout) == SFFN_ROPE_INTERLEAVED;
    a.norm = c->norm != 0;
    a.eps = c->eps;
    a.T = T;
    a.pos = positions;
    a.table = table;
    a.q_w = a.norm ? q_weight : nullptr;
    a.k_w = a.norm ? k_weight : nullptr;
    return a;
}

// ---- cache ---------------------------------------------------------------------------

sffn_status_t check_cache(const sffn_kv_cache_t* c, const sffn_kv_batch_t* b, int64_t T) {
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

sffn_status_t check_cache_pointers(const sffn_kv_cache_t* c, const sffn_kv_batch_t* b) {
    const void* ptrs[] = {c->keys, c->values, c->k_scale, c->v_scale};
    const char* names[] = {"keys", "values", "k_scale", "v_scale"};
    for (int i = 0; i < 4; ++i) {
        if (!ptrs[i]) return fail(SFFN_ERR_INVALID_ARG, "%s is null", names[i]);
        if (!aligned16(ptrs[i])) return fail(SFFN_ERR_INVALID_ARG, "%s is not 16-byte aligned", names[i]);
    }
    if (b->max_pages < 1) return fail(SFFN_ERR_INVALID_ARG, "max_pages must be positive (got %d)", b->max_pages);
    if (!b->kv_lens || !b->block_table)
        return fail(SFFN_ERR_INVALID_ARG, "block_table and kv_lens must not be null");
    for (const void* p : {(const void*)b->block_table, (const void*)b->kv_lens, (const void*)b->cu})
        if (reinterpret_cast<uintptr_t>(p) % 4 != 0)
            return fail(SFFN_ERR_INVALID_ARG, "block_table, kv_lens and cu must be 4-byte aligned");
    return SFFN_OK;
}

sffn::CacheArgs cache_args(const sffn_kv_cache_t* c, const sffn_kv_batch_t* b, int dtype, int64_t T) {
    sffn::CacheArgs a{};
    a.keys = c->keys;
    a.values = c->values;
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;
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
    a.dt = dtype == SFFN_BF16 ? sffn::Dt::BF16 : sffn::Dt::F32;
    return a;
}

typedef hipError_t (*CacheCopy)(const sffn::CacheArgs&, const sffn::Heads&, const sffn::Heads&, hipStream_t);

sffn_status_t cache_copy(const sffn_kv_cache_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* k,
                         const sffn_heads_t* v, const sffn_dtype_t& dtype, int64_t T, void* hip_stream, bool out,
                         CacheCopy launch, const char* what) {
    const int dt = as_int(dtype);
    SFFN_TRY(check_dtype(dt));
    SFFN_TRY(check_cache(cache, batch, T));
    if (T == 0 || batch->n_seqs == 0 || batch->max_new == 0) return SFFN_OK;
    SFFN_TRY(check_cache_pointers(cache, batch));
    SFFN_TRY(check_heads(k, "k", T, cache->kv_heads, cache->head_dim, dt, true, out));
    SFFN_TRY(check_heads(v, "v", T, cache->kv_heads, cache->head_dim, dt, true, out));
    const sffn::CacheArgs a = cache_args(cache, batch, dt, T);
    if (sffn::cache_copy_blocks(a) > kMaxGrid)
        return fail(SFFN_ERR_UNSUPPORTED, "T = %lld is too large for one call", (long long)T);
    return hip_status(launch(a, view(k), view(v), static_cast<hipStream_t>(hip_stream)), what);
}

// The checks of cache_attention that its workspace size needs too.
sffn_status_t check_attention(const sffn_kv_cache_t* cache, const sffn_kv_batch_t* batch, int32_t n_q_heads,
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

sffn_status_t make_plan(const sffn::CacheArgs& a, int32_t n_q_heads, int32_t window, sffn::AttnPlan* plan) {
    const int64_t tiles = ((int64_t)a.max_new * (n_q_heads / a.Hkv) + 15) / 16;
    if (tiles > kMaxGrid || (int64_t)a.B * a.Hkv > kMaxGrid / (tiles > 0 ? tiles : 1))
        return fail(SFFN_ERR_UNSUPPORTED, "the batch is too large for one call");
    // the kernels' counts of steps of 64 keys over all sequences and heads
    const int64_t steps = (int64_t)a.max_pages * a.P / 64 + 8;
    if ((int64_t)a.B * a.Hkv > kMaxGrid / steps)
        return fail(SFFN_ERR_UNSUPPORTED, "%d sequences of %d pages are too many for one call", a.B, a.max_pages);
    *plan = sffn::attn_plan(a, n_q_heads, window);
    if (plan->blocks > kMaxGrid) return fail(SFFN_ERR_UNSUPPORTED, "the batch is too large for one call");
    return SFFN_OK;
}

}  // namespace

extern "C" {

sffn_status_t qk_norm_rope(const sffn_rope_config_t* cfg, const sffn_heads_t* q, const sffn_heads_t* k,
                           const int32_t* positions, const float* table, const void* q_weight, const void* k_weight,
                           int64_t T, const sffn_heads_t* q_out, const sffn_heads_t* k_out, void* hip_stream) {
    SFFN_TRY(check_rope(cfg));
    if (T < 0) return fail(SFFN_ERR_INVALID_ARG, "T must be >= 0 (got %lld)", (long long)T);
    if (T == 0) return SFFN_OK;
    SFFN_TRY(check_rope_inputs(cfg, positions, table, q_weight, k_weight, T));
    const int dt = as_int(cfg->dtype);
    SFFN_TRY(check_heads(q, "q", T, cfg->n_q_heads, cfg->head_dim, dt, false, false));
    SFFN_TRY(check_heads(q_out, "q_out", T, cfg->n_q_heads, cfg->head_dim, dt, false, true));
    sffn::RopeArgs a = rope_args(cfg, positions, table, q_weight, k_weight, T);
    a.q = view(q);
    a.q_out = view(q_out);
    if (cfg->n_k_heads > 0) {
        SFFN_TRY(check_heads(k, "k", T, cfg->n_k_heads, cfg->head_dim, dt, false, false));
        SFFN_TRY(check_heads(k_out, "k_out", T, cfg->n_k_heads, cfg->head_dim, dt, false, true));
        a.k = view(k);
        a.k_out = view(k_out);
    }
    return hip_status(sffn::launch_rope(a, static_cast<hipStream_t>(hip_stream)), "qk_norm_rope");
}

size_t qk_norm_rope_backward_workspace_size(const sffn_rope_config_t* cfg, int64_t T) {
    if (check_rope(cfg) != SFFN_OK || T <= 0) return 0;
    return sffn::rope_partial_floats(rope_args(cfg, nullptr, nullptr, nullptr, nullptr, T)) * 4;
}

sffn_status_t qk_norm_rope_backward(const sffn_rope_config_t* cfg, const sffn_heads_t* q, const sffn_heads_t* k,
                                    const sffn_heads_t* g_q, const sffn_heads_t* g_k, const int32_t* positions,
                                    const float* table, const void* q_weight, const void* k_weight, int64_t T,
                                    const sffn_heads_t* g_q_in, const sffn_heads_t* g_k_in, float* g_q_weight,
                                    float* g_k_weight, void* workspace, size_t ws_bytes, void* hip_stream) {
    SFFN_TRY(check_rope(cfg));
    if (T < 0) return fail(SFFN_ERR_INVALID_ARG, "T must be >= 0 (got %lld)", (long long)T);
    if (reinterpret_cast<uintptr_t>(g_q_weight) % 4 != 0 || reinterpret_cast<uintptr_t>(g_k_weight) % 4 != 0)
        return fail(SFFN_ERR_INVALID_ARG, "the weights' gradients must be 4-byte aligned");
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (T == 0) {
        hipError_t he = hipSuccess;
        for (float* p : {g_q_weight, g_k_weight})
            if (he == hipSuccess && p && cfg->norm) he = sffn::launch_zero_f32(p, cfg->head_dim, s);
        return hip_status(he, "qk_norm_rope_backward");
    }
    SFFN_TRY(check_rope_inputs(cfg, positions, table, q_weight, k_weight, T));
    const int dt = as_int(cfg->dtype), D = cfg->head_dim;
    sffn::RopeArgs a = rope_args(cfg, positions, table, q_weight, k_weight, T);
    if (a.norm) SFFN_TRY(check_heads(q, "q", T, cfg->n_q_heads, D, dt, false, false));
    SFFN_TRY(check_heads(g_q, "g_q", T, cfg->n_q_heads, D, dt, false, false));
    SFFN_TRY(check_heads(g_q_in, "g_q_in", T, cfg->n_q_heads, D, dt, false, true));
    a.g_q = view(g_q);
    a.q_out = view(g_q_in);
    if (a.norm) a.q = view(q);
    if (cfg->n_k_heads > 0) {
        if (a.norm) SFFN_TRY(check_heads(k, "k", T, cfg->n_k_heads, D, dt, false, false));
        SFFN_TRY(check_heads(g_k, "g_k", T, cfg->n_k_heads, D, dt, false, false));
        SFFN_TRY(check_heads(g_k_in, "g_k_in", T, cfg->n_k_heads, D, dt, false, true));
        a.g_k = view(g_k);
        a.k_out = view(g_k_in);
        if (a.norm) a.k = view(k);
    }
    if (a.norm && (g_q_weight || g_k_weight)) {
        const size_t need = sffn::rope_partial_floats(a) * 4;
        if (!workspace) return fail(SFFN_ERR_INVALID_ARG, "workspace is null");
        if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
            return fail(SFFN_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
        if (ws_bytes < need)
            return fail(SFFN_ERR_WORKSPACE, "workspace holds %zu bytes, %zu needed", ws_bytes, need);
        a.partial = static_cast<float*>(workspace);
        a.g_qw = g_q_weight;
        a.g_kw = g_k_weight;
    }
    return hip_status(sffn::launch_rope_backward(a, s), "qk_norm_rope_backward");
}

sffn_status_t kv_cache_append(const sffn_kv_cache_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* k,
                              const sffn_heads_t* v, sffn_dtype_t dtype, int64_t T, void* hip_stream) {
    return cache_copy(cache, batch, k, v, dtype, T, hip_stream, false, sffn::launch_cache_append, "kv_cache_append");
}

sffn_status_t kv_cache_read(const sffn_kv_cache_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* k,
                            const sffn_heads_t* v, sffn_dtype_t dtype, int64_t T, void* hip_stream) {
    return cache_copy(cache, batch, k, v, dtype, T, hip_stream, true, sffn::launch_cache_read, "kv_cache_read");
}

size_t cache_attention_workspace_size(const sffn_kv_cache_t* cache, const sffn_kv_batch_t* batch, int32_t n_q_heads,
                                      sffn_dtype_t dtype, int32_t window, int64_t T) {
    if (check_dtype(as_int(dtype)) != SFFN_OK || check_attention(cache, batch, n_q_heads, window, T) != SFFN_OK) return 0;
    if (T == 0 || batch->n_seqs == 0 || batch->max_new == 0) return 0;
    sffn::AttnPlan plan;
    if (make_plan(cache_args(cache, batch, as_int(dtype), T), n_q_heads, window, &plan) != SFFN_OK) return 0;
    return plan.ws_bytes;
}

sffn_status_t cache_attention(const sffn_kv_cache_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* q,
                              int32_t n_q_heads, sffn_dtype_t dtype, int64_t T, float scale, int32_t window,
                              const sffn_heads_t* out, float* lse, void* workspace, size_t ws_bytes,
                              void* hip_stream) {
    const int dt = as_int(dtype);
    SFFN_TRY(check_dtype(dt));
    SFFN_TRY(check_attention(cache, batch, n_q_heads, window, T));
    if (!std::isfinite(scale)) return fail(SFFN_ERR_INVALID_ARG, "scale must be finite (got %g)", (double)scale);
    if (T == 0 || batch->n_seqs == 0 || batch->max_new == 0) return SFFN_OK;
    SFFN_TRY(check_cache_pointers(cache, batch));
    SFFN_TRY(check_heads(q, "q", T, n_q_heads, cache->head_dim, dt, true, false));
    SFFN_TRY(check_heads(out, "out", T, n_q_heads, cache->head_dim, dt, true, true));
    if (reinterpret_cast<uintptr_t>(lse) % 4 != 0) return fail(SFFN_ERR_INVALID_ARG, "lse must be 4-byte aligned");
    const sffn::CacheArgs a = cache_args(cache, batch, dt, T);
    sffn::AttnPlan plan;
    SFFN_TRY(make_plan(a, n_q_heads, window, &plan));
    if (plan.ws_bytes > 0) {
        if (!workspace) return fail(SFFN_ERR_INVALID_ARG, "workspace is null");
        if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
            return fail(SFFN_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
        if (ws_bytes < plan.ws_bytes)
            return fail(SFFN_ERR_WORKSPACE, "workspace holds %zu bytes, %zu needed", ws_bytes, plan.ws_bytes);
    }
    return hip_status(sffn::launch_cache_attention(a, plan, view(q), n_q_heads, scale, window, view(out), lse,
                                                   workspace, static_cast<hipStream_t>(hip_stream)),
                      "cache_attention");
}

}  // extern "C"
