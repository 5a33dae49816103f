// C ABI of the page bookkeeping (include/sparse_ffn_paging.h): argument checks and the
// calls of the launchers.
#include <hip/hip_runtime.h>

#include "../../include/sparse_ffn_paging.h"
#include "paging_launch.hpp"
#include "status.hpp"

namespace {

using sffn::fail;
using sffn::hip_status;

constexpr int64_t kMaxNewTokens = (int64_t)1 << 28;     // as the cache's own calls take
constexpr int64_t kMaxCapacity = (int64_t)1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 42;
constexpr int32_t kMaxSeqs = 1 << 24;

#define SFFN_TRY(call)                        \
    do {                                      \
        const sffn_status_t try_st = (call);  \
        if (try_st != SFFN_OK) return try_st; \
    } while (0)

sffn_status_t check_tables(int64_t table_stride, int64_t n_pages, int32_t n_seqs, int32_t max_pages, int32_t page,
                           int64_t T) {
    if (page != 16 && page != 32 && page != 64 && page != 128)
        return fail(SFFN_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128 (got %d)", page);
    if (n_pages < 1 || n_pages > INT32_MAX)
        return fail(SFFN_ERR_INVALID_ARG, "n_pages must lie in [1, 2^31) (got %lld)", (long long)n_pages);
    if (n_seqs < 0 || n_seqs > kMaxSeqs)
        return fail(SFFN_ERR_INVALID_ARG, "n_seqs must lie in [0, 2^24] (got %d)", n_seqs);
    if (max_pages < 1) return fail(SFFN_ERR_INVALID_ARG, "max_pages must be positive (got %d)", max_pages);
    if ((int64_t)max_pages * page > kMaxCapacity)
        return fail(SFFN_ERR_UNSUPPORTED, "max_pages %d of %d tokens are too many", max_pages, page);
    if (table_stride < 0 || table_stride > kMaxStride || (n_seqs > 1 && table_stride < max_pages))
        return fail(SFFN_ERR_INVALID_ARG, "table_stride %lld does not fit rows of %d pages", (long long)table_stride,
                    max_pages);
    if (T < 0) return fail(SFFN_ERR_INVALID_ARG, "T must be >= 0 (got %lld)", (long long)T);
    if (T > kMaxNewTokens) return fail(SFFN_ERR_UNSUPPORTED, "T = %lld is too large for one call", (long long)T);
    return SFFN_OK;
}

sffn_status_t check_pointer(const void* p, const char* name, size_t e, bool needed) {
    if (!p && needed) return fail(SFFN_ERR_INVALID_ARG, "%s is null", name);
    if (reinterpret_cast<uintptr_t>(p) % e != 0)
        return fail(SFFN_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
    return SFFN_OK;
}

}  // namespace

extern "C" {

sffn_status_t page_plan(const sffn_page_pool_t* pool, const int32_t* kv_lens, const int32_t* keep_lens,
                        const int32_t* new_lens, const int32_t* n_free, int64_t T, int32_t* kv_lens_out,
                        int32_t* n_free_out, int32_t* cu, int32_t* positions, int64_t* slots, void* hip_stream) {
    if (!pool) return fail(SFFN_ERR_INVALID_ARG, "pool is null");
    SFFN_TRY(check_tables(pool->table_stride, pool->n_pages, pool->n_seqs, pool->max_pages, pool->page, T));
    const bool any = pool->n_seqs > 0;
    SFFN_TRY(check_pointer(pool->block_table, "block_table", 4, any));
    SFFN_TRY(check_pointer(pool->free_pages, "free_pages", 4, true));
    SFFN_TRY(check_pointer(kv_lens, "kv_lens", 4, any));
    SFFN_TRY(check_pointer(keep_lens, "keep_lens", 4, false));
    SFFN_TRY(check_pointer(new_lens, "new_lens", 4, any));
    SFFN_TRY(check_pointer(n_free, "n_free", 4, true));
    SFFN_TRY(check_pointer(kv_lens_out, "kv_lens_out", 4, any));
    SFFN_TRY(check_pointer(n_free_out, "n_free_out", 4, true));
    SFFN_TRY(check_pointer(cu, "cu", 4, true));
    SFFN_TRY(check_pointer(positions, "positions", 4, T > 0));
    SFFN_TRY(check_pointer(slots, "slots", 8, T > 0));
    if (any && (kv_lens_out == keep_lens || kv_lens_out == new_lens))
        return fail(SFFN_ERR_INVALID_ARG, "kv_lens_out may be kv_lens alone of the inputs");
    sffn::PlanArgs a{};
    a.table = pool->block_table;
    a.table_stride = pool->table_stride;
    a.free_pages = pool->free_pages;
    a.n_pages = pool->n_pages;
    a.T = T;
    a.B = pool->n_seqs;
    a.max_pages = pool->max_pages;
    a.shift = __builtin_ctz((unsigned)pool->page);
    a.lens = kv_lens;
    a.keep = keep_lens;
    a.fresh = new_lens;
    a.n_free = n_free;
    a.lens_out = kv_lens_out;
    a.n_free_out = n_free_out;
    a.cu = cu;
    a.positions = positions;
    a.slots = slots;
    return hip_status(sffn::launch_page_plan(a, static_cast<hipStream_t>(hip_stream)), "page_plan");
}

sffn_status_t cache_slots(const sffn_kv_batch_t* batch, int64_t n_pages, int32_t page, int64_t T, int32_t* positions,
                          int64_t* slots, void* hip_stream) {
    if (!batch) return fail(SFFN_ERR_INVALID_ARG, "batch is null");
    SFFN_TRY(check_tables(batch->table_stride, n_pages, batch->n_seqs, batch->max_pages, page, T));
    if (batch->max_new < 0) return fail(SFFN_ERR_INVALID_ARG, "max_new must not be negative");
    if (!batch->cu && T != batch->n_seqs)
        return fail(SFFN_ERR_INVALID_ARG, "without cu, T must be n_seqs (got %lld, %d)", (long long)T, batch->n_seqs);
    if (T == 0) return SFFN_OK;
    const bool any = batch->n_seqs > 0;
    SFFN_TRY(check_pointer(batch->block_table, "block_table", 4, any));
    SFFN_TRY(check_pointer(batch->kv_lens, "kv_lens", 4, any));
    SFFN_TRY(check_pointer(batch->cu, "cu", 4, false));
    SFFN_TRY(check_pointer(positions, "positions", 4, true));
    SFFN_TRY(check_pointer(slots, "slots", 8, true));
    sffn::SlotArgs a{};
    a.table = batch->block_table;
    a.table_stride = batch->table_stride;
    a.lens = batch->kv_lens;
    a.cu = batch->cu;
    a.B = batch->n_seqs;
    a.max_pages = batch->max_pages;
    a.max_new = batch->max_new;
    a.shift = __builtin_ctz((unsigned)page);
    a.n_pages = n_pages;
    a.T = T;
    a.positions = positions;
    a.slots = slots;
    return hip_status(sffn::launch_slots(a, static_cast<hipStream_t>(hip_stream)), "cache_slots");
}

}  // extern "C"
