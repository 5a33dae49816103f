/*
 * sparse_ffn_attention.h -- C ABI of the attention-side operators of a decoder
 * layer that stand next to the sparse FFN (AMD Instinct MI355X, gfx950):
 *
 *   qk_norm_rope           norms of q and k for each head and the rotation of
 *   qk_norm_rope_backward  their pairs by position, in one pass; its gradient
 *   kv_cache_append        new keys and values into a paged 8-bit cache
 *   kv_cache_read          tokens of the cache as the values they stand for
 *   cache_attention        attention of new tokens over that cache
 *   kv_cache4_append, kv_cache4_read, cache4_attention
 *                          the same for a paged 4-bit cache
 *
 * The conventions of sparse_ffn.h hold: status codes only, every argument
 * checked before anything is enqueued, asynchronous on `hip_stream`, nothing
 * allocated, bf16 as uint16 storage, sparse_ffn_last_error() for the detail.
 * Sizes and pointers are checked on the host. Values held in device memory
 * (positions, block tables, lengths) are not known there: the kernels bound
 * every address they form from them, and an entry out of range shows as NaN in
 * the rows that use it (kv_cache_append: the tokens concerned are not stored).
 */
#ifndef SPARSE_FFN_ATTENTION_H
#define SPARSE_FFN_ATTENTION_H

#include "sparse_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A [T, heads, head_dim] view: element (t, h, i) lies at data + t stride_token
 * + h stride_head + i (strides in elements, >= 0; the last dimension is
 * contiguous). Outputs must not overlap themselves. */
typedef struct {
    void* data;             /* device; const where the view is an input */
    int64_t stride_token;
    int64_t stride_head;
} sffn_heads_t;

/* ---- head norms and rotary positions -------------------------------------- */

typedef enum {
    SFFN_ROPE_HALF = 0,        /* pairs (i, i + rot_dim / 2) */
    SFFN_ROPE_INTERLEAVED = 1  /* pairs (2 i, 2 i + 1)       */
} sffn_rope_layout_t;

/* n_q_heads >= 1, n_k_heads >= 0 (0: q alone), both <= 65536; 1 <= head_dim
 * <= 512; rot_dim even, 0 <= rot_dim <= head_dim (elements from rot_dim on are
 * not rotated); eps > 0 with norm; max_pos >= 1 rows of the table. */
typedef struct {
    int32_t n_q_heads;
    int32_t n_k_heads;
    int32_t head_dim;
    int32_t rot_dim;
    int32_t max_pos;
    sffn_dtype_t dtype;        /* of q, k, the weights, outputs and their gradients */
    sffn_rope_layout_t layout;
    int32_t norm;              /* 0: rotation alone; 1: RMS norm of every head first */
    float eps;
} sffn_rope_config_t;

/* For every token t and head (fp32 inside, one rounding at the end):
 *   n = x * rsqrt(mean(x^2) + eps) * w        (norm = 0: n = x)
 *   y_a = n_a c - n_b s,  y_b = n_b c + n_a s for pair i = (a, b), with
 *   c = table[positions[t]][i], s = table[positions[t]][rot_dim / 2 + i]
 *   q, q_out, k, k_out  [T, heads, head_dim] views; an output may be its own
 *                       input (same data and strides). k and k_out may be NULL
 *                       with n_k_heads = 0
 *   positions [T] int32, table [max_pos, rot_dim] fp32: cos | sin (device). A
 *             position outside [0, max_pos) makes that token's rows NaN. Both
 *             may be NULL with rot_dim = 0
 *   q_weight, k_weight [head_dim] or NULL (ones), read with norm only
 * T == 0 enqueues nothing. */
sffn_status_t qk_norm_rope(const sffn_rope_config_t* cfg, const sffn_heads_t* q, const sffn_heads_t* k,
                           const int32_t* positions, const float* table, const void* q_weight,
                           const void* k_weight, int64_t T, const sffn_heads_t* q_out,
                           const sffn_heads_t* k_out, void* hip_stream);

/* Workspace bytes of qk_norm_rope_backward (0 when the config is invalid, T <=
 * 0, or without norm, which needs none). */
size_t qk_norm_rope_backward_workspace_size(const sffn_rope_config_t* cfg, int64_t T);

/* Gradients of L for gradients g_q, g_k of qk_norm_rope's outputs; q and k are
 * that call's inputs (read with norm only: NULL otherwise allowed). g_q_in and
 * g_k_in receive dL/dq and dL/dk (cfg->dtype) and may be g_q and g_k
 * themselves; g_q_weight, g_k_weight [head_dim] fp32 receive the weights'
 * gradients, summed over tokens and heads in a fixed order (NULL: not wanted;
 * ignored without norm; zeros for T == 0). */
sffn_status_t qk_norm_rope_backward(const sffn_rope_config_t* cfg, const sffn_heads_t* q, const sffn_heads_t* k,
                                    const sffn_heads_t* g_q, const sffn_heads_t* g_k, const int32_t* positions,
                                    const float* table, const void* q_weight, const void* k_weight, int64_t T,
                                    const sffn_heads_t* g_q_in, const sffn_heads_t* g_k_in, float* g_q_weight,
                                    float* g_k_weight, void* workspace, size_t ws_bytes, void* hip_stream);

/* ---- the 8-bit cache --------------------------------------------------------- */

/* A pool of pages of `page` tokens for each of kv_heads heads. A key or value
 * is its int8 entry times the scale of its page and head.
 *   keys     int8 [n_pages, kv_heads, page, head_dim]
 *   values   int8 [n_pages, kv_heads, head_dim, page] (a channel's tokens are
 *            contiguous: the order the matrix cores take them in)
 *   k_scale, v_scale  fp32 [n_pages, kv_heads], not negative
 * page 16, 32, 64 or 128; head_dim 64, 128 or 256; pointers 16-byte aligned. */
typedef struct {
    int8_t* keys;
    int8_t* values;
    float* k_scale;
    float* v_scale;
    int64_t n_pages;
    int32_t kv_heads;
    int32_t page;
    int32_t head_dim;
} sffn_kv_cache_t;

/* Sequences and the tokens of this call: sequence b holds kv_lens[b] tokens in
 * the pages block_table[b][0 ..]; the call's tokens cu[b] .. cu[b + 1] - 1 are
 * its last ones (their keys and values included in kv_lens). With cu NULL
 * token b is the last token of sequence b.
 *   block_table [n_seqs] rows of max_pages int32 (row stride table_stride);
 *               max_pages * page at most 2^30, T at most 2^28
 *   kv_lens [n_seqs] int32, cu [n_seqs + 1] int32 ascending from 0, or NULL
 *   max_new   >= every cu[b + 1] - cu[b] (T always is); it splits the work. Tokens
 *             of a sequence beyond its first max_new are not stored by an append;
 *             a read and attention make their rows NaN, as they do with all rows
 *             of a sequence whose offsets leave the call
 *   max_kv    about the largest kv_lens[b]: splits the work, never the result */
typedef struct {
    const int32_t* block_table;
    int64_t table_stride;
    const int32_t* kv_lens;
    const int32_t* cu;
    int32_t n_seqs;
    int32_t max_pages;
    int32_t max_new;
    int32_t max_kv;
} sffn_kv_batch_t;

/* Store k, v [T, kv_heads, head_dim] (views, 16-byte aligned rows) of the
 * batch's tokens. For every page and head that receives tokens, with old
 * entries q and scale s where the page held tokens of the sequence before:
 *   s' = max(s, max|x| / 127) over the new x (s' = max|x| / 127 in a page that
 *        held none),  q' = rint(q (s / s')),  new entries rint(x / s'),
 * so that no entry leaves [-127, 127]. A page and head that receives a NaN or
 * an infinity gets scale NaN. Two sequences must not append to one page. */
sffn_status_t kv_cache_append(const sffn_kv_cache_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* k,
                              const sffn_heads_t* v, sffn_dtype_t dtype, int64_t T, void* hip_stream);

/* The batch's tokens out of the cache: entry times scale, rounded to dtype, to
 * k, v [T, kv_heads, head_dim] (views, 16-byte aligned rows). */
sffn_status_t kv_cache_read(const sffn_kv_cache_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* k,
                            const sffn_heads_t* v, sffn_dtype_t dtype, int64_t T, void* hip_stream);

/* Workspace bytes of cache_attention for T tokens of n_q_heads heads (0 when
 * an argument is invalid or none is needed; 256 MiB at most). */
size_t cache_attention_workspace_size(const sffn_kv_cache_t* cache, const sffn_kv_batch_t* batch,
                                      int32_t n_q_heads, sffn_dtype_t dtype, int32_t window, int64_t T);

/* Attention of the batch's tokens over the cache. Token i of sequence b's n
 * new ones stands at position p = kv_lens[b] - n + i and sees the keys j with
 * p - window < j <= p (window 0: every j <= p); query head a reads the keys and
 * values of head a / (n_q_heads / kv_heads):
 *   s_j = scale q . k_j,  out = sum_j softmax(s)_j v_j,  lse = log sum_j exp s_j
 * Scores, statistics and sums are fp32; the weights of the values are kept to
 * fp32 for an fp32 q. For a bf16 q they are kept to 16 bits in a sequence of up
 * to 128 rows (new tokens times n_q_heads / kv_heads) and to 8 (bf16) in one of
 * more, whatever the call's other sequences and max_new. A row that sees no key
 * gives zeros and lse -inf.
 *   q, out [T, n_q_heads, head_dim] views (dtype, 16-byte aligned rows); rows
 *          of tokens outside every sequence are left as they are
 *   lse    [T, n_q_heads] fp32 or NULL (device)
 *   n_q_heads a multiple of kv_heads; window >= 0; scale finite
 *   workspace  as for sparse_ffn_forward; may be NULL when its size is 0 */
sffn_status_t cache_attention(const sffn_kv_cache_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* q,
                              int32_t n_q_heads, sffn_dtype_t dtype, int64_t T, float scale, int32_t window,
                              const sffn_heads_t* out, float* lse, void* workspace, size_t ws_bytes,
                              void* hip_stream);

/* ---- the 4-bit cache --------------------------------------------------------- */

/* As the 8-bit cache, with entries of 4-bit floating point: a sign, two bits of exponent
 * and one of mantissa, the codes 0 .. 7 standing for 0, 0.5, 1, 1.5, 2, 3, 4, 6 and 8 .. 15
 * for their negatives; two in a byte, the even channel in the low half. Every token's
 * scales are its own, so an append changes no other token's entries.
 *   keys, values  uint8 [n_pages, kv_heads, page, head_dim / 2]
 *   k_exp    uint8 [n_pages, kv_heads, page, head_dim / 32]: a key is its entry times
 *            2^(k_exp - 127) of its 32 channels; 255 stands for NaN
 *   v_scale  fp32 [n_pages, kv_heads, page], not negative: a value is its entry times its
 *            token's scale
 * page 16, 32, 64 or 128; head_dim 64, 128 or 256; pointers 16-byte aligned. 68 + 68 bytes
 * a token and head of 128 channels, where the 8-bit cache takes 256. */
typedef struct {
    uint8_t* keys;
    uint8_t* values;
    uint8_t* k_exp;
    float* v_scale;
    int64_t n_pages;
    int32_t kv_heads;
    int32_t page;
    int32_t head_dim;
} sffn_kv_cache4_t;

/* Store k, v [T, kv_heads, head_dim] (views, 16-byte aligned rows) of T tokens. For each 32
 * channels of a key the least power of two by which none of them exceeds 6 (at least
 * 2^-127), and 255 where one is NaN or infinite; for a value v_scale = max|v| / 6 (NaN where
 * one is NaN or infinite). Entries are x / scale rounded to the nearest, ties to the even
 * code (IEEE fp32 arithmetic; zero where v_scale is 0, undefined where a scale is NaN).
 *   slots  [T] int64 (device): page * (page's number) + (place in the page) of every token,
 *          which is not stored where that lies outside the pool; NULL: the slots follow from
 *          the batch. With slots the batch may be NULL, and nothing of it is read but its
 *          offsets and max_new: where it has cu, tokens beyond max_new of their sequence are
 *          not stored, as without slots. No two tokens may have the same slot. */
sffn_status_t kv_cache4_append(const sffn_kv_cache4_t* cache, const sffn_kv_batch_t* batch, const int64_t* slots,
                               const sffn_heads_t* k, const sffn_heads_t* v, sffn_dtype_t dtype, int64_t T,
                               void* hip_stream);

/* As kv_cache_read. */
sffn_status_t kv_cache4_read(const sffn_kv_cache4_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* k,
                             const sffn_heads_t* v, sffn_dtype_t dtype, int64_t T, void* hip_stream);

/* As cache_attention_workspace_size and cache_attention. The products take 4-bit entries as
 * they are; q and the weights of the values are sums of 6-bit pieces relative to the largest
 * of 32 channels (q) or keys (weights). A bf16 q: its entries, those below 2^-10 of the largest
 * to 2^-17.9 of it; in sequences of more than 128 rows a key head, heads of 64 and 256: its
 * products with the scale to 2^-17.9. Weights: to 2^-13.9, in sequences of more than 128 rows to
 * 2^-7.9 (to 2^-9 below a quarter of the largest). An fp32 q and its weights: to 2^-21.9.
 * Sums are fp32, of weights up to 2^8: finite where a sequence's keys times its largest value
 * stay below 2^120. */
size_t cache4_attention_workspace_size(const sffn_kv_cache4_t* cache, const sffn_kv_batch_t* batch,
                                       int32_t n_q_heads, sffn_dtype_t dtype, int32_t window, int64_t T);
sffn_status_t cache4_attention(const sffn_kv_cache4_t* cache, const sffn_kv_batch_t* batch, const sffn_heads_t* q,
                               int32_t n_q_heads, sffn_dtype_t dtype, int64_t T, float scale, int32_t window,
                               const sffn_heads_t* out, float* lse, void* workspace, size_t ws_bytes,
                               void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_FFN_ATTENTION_H */
