/*
 * sparse_ffn_paging.h -- C ABI of the page bookkeeping of a paged cache on the GPU (AMD
 * Instinct MI355X, gfx950): which pages a step's tokens go to, without a copy to the host.
 *
 *   page_plan    of the requests of a step: pages given back and taken, lengths, offsets,
 *                and of every new token its position and slot
 *   cache_slots  positions and slots of the new tokens of a batch that is there already
 *
 * The conventions of sparse_ffn.h and sparse_ffn_attention.h hold. The slot of a token is
 * page * (its page's number) + (its place in the page): its row in a cache laid out
 * [pages, page, ...], the same for every layer of a model. -1: the token has none.
 */
#ifndef SPARSE_FFN_PAGING_H
#define SPARSE_FFN_PAGING_H

#include "sparse_ffn_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Block tables and the pages that no sequence holds.
 *   block_table [n_seqs] rows of max_pages int32 (row stride table_stride), in place
 *   free_pages  [n_pages] int32, in place: a stack, of which the first n_free[0] count
 *   page        16, 32, 64 or 128 tokens; max_pages * page at most 2^30
 *   n_seqs at most 2^24, n_pages below 2^31 */
typedef struct {
    int32_t* block_table;
    int64_t table_stride;
    int32_t* free_pages;
    int64_t n_pages;
    int32_t n_seqs;
    int32_t max_pages;
    int32_t page;
} sffn_page_pool_t;

/* The next step of every sequence b, which holds kv_lens[b] tokens: it keeps the first
 * min(kv_lens[b], keep_lens[b]) of them (keep_lens NULL: all; 0 ends a sequence, a few less
 * than kv_lens takes refused drafts back) and gets new_lens[b] more (numbers below zero count as
 * zero; together fewer than 2^31):
 *   kv_lens_out[b]  tokens held then;  cu[0 .. n_seqs] offsets of the new ones
 *   free_pages, block_table  pages behind those kept go onto the stack, in the order of
 *       sequences and of their pages (entries that name no page are passed over); then the
 *       pages of the new tokens come off its top in the same order. Where none is left
 *       the entry is -1. Tokens behind max_pages pages have no page.
 *   n_free_out[0]   pages left on the stack, [1] pages that this call lacked
 *   positions [T] int32, slots [T] int64 of the new tokens (the call's size T bounds what is
 *       written; tokens behind the last sequence's have position 0 and slot -1)
 * kv_lens_out may be kv_lens and n_free_out n_free; no other two may overlap. */
sffn_status_t page_plan(const sffn_page_pool_t* pool, const int32_t* kv_lens, const int32_t* keep_lens,
                        const int32_t* new_lens, const int32_t* n_free, int64_t T, int32_t* kv_lens_out,
                        int32_t* n_free_out, int32_t* cu, int32_t* positions, int64_t* slots, void* hip_stream);

/* Positions and slots of the T new tokens of a batch (see sffn_kv_batch_t) whose tables are
 * filled. Tokens of no sequence, beyond their sequence's first max_new, or of a sequence whose
 * offsets leave the call have slot -1 (those of no sequence position 0). */
sffn_status_t cache_slots(const sffn_kv_batch_t* batch, int64_t n_pages, int32_t page, int64_t T, int32_t* positions,
                          int64_t* slots, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_FFN_PAGING_H */
