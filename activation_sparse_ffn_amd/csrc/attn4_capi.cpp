// C ABI of the 4-bit cache (include/sparse_ffn_attention.h): argument checks, workspace
// sizes and the calls of the launchers.
#include <hip/hip_runtime.h>

#include <cmath>

#include "attn_checks.hpp"

namespace {

using namespace sffn;

CacheBuffers buffers(const sffn_kv_cache4_t* c) {
    return {{c->keys, c->values, c->k_exp, c->v_scale}, {"keys", "values", "k_exp", "v_scale"}};
}

Cache4 cache4(const sffn_kv_cache4_t* c) { return {c->keys, c->values, c->k_exp, c->v_scale}; }

// Of an append by slots: of the batch, where there is one, offsets and max_new are read.
sffn_status_t check_slots(const int64_t* slots, const sffn_kv_batch_t* batch) {
    if (!slots) return SFFN_OK;
    if (reinterpret_cast<uintptr_t>(slots) % 8 != 0)
        return fail(SFFN_ERR_INVALID_ARG, "slots must be 8-byte aligned");
    if (!batch) return SFFN_OK;
    if (batch->n_seqs < 0 || batch->max_new < 0)
        return fail(SFFN_ERR_INVALID_ARG, "n_seqs and max_new must not be negative");
    if (reinterpret_cast<uintptr_t>(batch->cu) % 4 != 0)
        return fail(SFFN_ERR_INVALID_ARG, "cu must be 4-byte aligned");
    return SFFN_OK;
}

sffn_status_t check_copy(const sffn_kv_cache4_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* k,
                         const sffn_heads_t* v, int dt, int64_t T, bool out) {
    SFFN_TRY(check_cache_pointers(buffers(cache), batch));
    SFFN_TRY(check_heads(k, "k", T, cache->kv_heads, cache->head_dim, dt, true, out));
    SFFN_TRY(check_heads(v, "v", T, cache->kv_heads, cache->head_dim, dt, true, out));
    if (T * cache->kv_heads > kMaxGrid)
        return fail(SFFN_ERR_UNSUPPORTED, "T = %lld is too large for one call", (long long)T);
    return SFFN_OK;
}

}  // namespace

extern "C" {

sffn_status_t kv_cache4_append(const sffn_kv_cache4_t* cache, const sffn_kv_batch_t* batch, const int64_t* slots,
                               const sffn_heads_t* k, const sffn_heads_t* v, sffn_dtype_t dtype, int64_t T,
                               void* hip_stream) {
    const int dt = as_int(dtype);
    SFFN_TRY(check_dtype(dt));
    SFFN_TRY(check_slots(slots, batch));
    // the sequences that a call by slots stands for: as many as it has tokens, a page each
    sffn_kv_batch_t by_slots{};
    int32_t unused = 0;
    // which matters where one can have more than max_new of them
    const sffn_kv_batch_t* given = slots && batch && batch->cu && batch->max_new < T ? batch : nullptr;
    if (slots) {
        if (T < 0 || T > INT32_MAX) return fail(SFFN_ERR_INVALID_ARG, "T must lie in [0, 2^31) (got %lld)", (long long)T);
        by_slots.n_seqs = (int32_t)T;
        by_slots.max_pages = 1;
        by_slots.table_stride = 1;
        by_slots.max_new = 1;
        by_slots.block_table = by_slots.kv_lens = &unused;
        batch = &by_slots;
    }
    SFFN_TRY(check_cache(cache, batch, T));
    if (T == 0 || batch->n_seqs == 0 || batch->max_new == 0) return SFFN_OK;
    if (given && given->max_new == 0) return SFFN_OK;
    SFFN_TRY(check_copy(cache, batch, k, v, dt, T, false));
    CacheArgs a = cache_shape(cache, batch, dt, T);
    if (slots) a.table = a.lens = nullptr;      // not read
    if (given && given->n_seqs > 0) {
        a.cu = given->cu;
        a.B = given->n_seqs;
        a.max_new = given->max_new;
    }
    return hip_status(launch_cache4_append(a, cache4(cache), slots, view(k), view(v), static_cast<hipStream_t>(hip_stream)),
                      "kv_cache4_append");
}

sffn_status_t kv_cache4_read(const sffn_kv_cache4_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* k,
                             const sffn_heads_t* v, sffn_dtype_t dtype, int64_t T, void* hip_stream) {
    const int dt = as_int(dtype);
    SFFN_TRY(check_dtype(dt));
    SFFN_TRY(check_cache(cache, batch, T));
    if (T == 0 || batch->n_seqs == 0 || batch->max_new == 0) return SFFN_OK;
    SFFN_TRY(check_copy(cache, batch, k, v, dt, T, true));
    return hip_status(launch_cache4_read(cache_shape(cache, batch, dt, T), cache4(cache), view(k), view(v),
                                         static_cast<hipStream_t>(hip_stream)),
                      "kv_cache4_read");
}

size_t cache4_attention_workspace_size(const sffn_kv_cache4_t* cache, const sffn_kv_batch_t* batch,
                                       int32_t n_q_heads, sffn_dtype_t dtype, int32_t window, int64_t T) {
    if (check_dtype(as_int(dtype)) != SFFN_OK || check_attention(cache, batch, n_q_heads, window, T) != SFFN_OK) return 0;
    if (T == 0 || batch->n_seqs == 0 || batch->max_new == 0) return 0;
    AttnPlan plan;
    if (make_plan(cache_shape(cache, batch, as_int(dtype), T), n_q_heads, window, attn4_plan, &plan, kUnitCost4) != SFFN_OK) return 0;
    return plan.ws_bytes;
}

sffn_status_t cache4_attention(const sffn_kv_cache4_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* q,
                               int32_t n_q_heads, sffn_dtype_t dtype, int64_t T, float scale, int32_t window,
                               const sffn_heads_t* out, float* lse, void* workspace, size_t ws_bytes,
                               void* hip_stream) {
    const int dt = as_int(dtype);
    SFFN_TRY(check_dtype(dt));
    SFFN_TRY(check_attention(cache, batch, n_q_heads, window, T));
    if (!std::isfinite(scale)) return fail(SFFN_ERR_INVALID_ARG, "scale must be finite (got %g)", (double)scale);
    if (T == 0 || batch->n_seqs == 0 || batch->max_new == 0) return SFFN_OK;
    SFFN_TRY(check_cache_pointers(buffers(cache), batch));
    SFFN_TRY(check_heads(q, "q", T, n_q_heads, cache->head_dim, dt, true, false));
    SFFN_TRY(check_heads(out, "out", T, n_q_heads, cache->head_dim, dt, true, true));
    if (reinterpret_cast<uintptr_t>(lse) % 4 != 0) return fail(SFFN_ERR_INVALID_ARG, "lse must be 4-byte aligned");
    const CacheArgs a = cache_shape(cache, batch, dt, T);
    AttnPlan plan;
    SFFN_TRY(make_plan(a, n_q_heads, window, attn4_plan, &plan, kUnitCost4));
    SFFN_TRY(check_workspace(workspace, ws_bytes, plan.ws_bytes));
    return hip_status(launch_cache4_attention(a, cache4(cache), plan, view(q), n_q_heads, scale, window, view(out), lse,
                                              workspace, static_cast<hipStream_t>(hip_stream)),
                      "cache4_attention");
}

}  // extern "C"
