/*
 * sparse_ffn_norm.h -- C ABI of the root-mean-square norm between the halves of a
 * decoder layer (AMD Instinct MI355X, gfx950):
 *
 *   add_rms_norm           the residual's addition and the norm in one pass, its
 *                          output in the input's type or in 8 bits with row scales
 *   add_rms_norm_backward  its gradient
 *
 * The conventions of sparse_ffn.h hold: status codes only, every argument checked
 * before anything is enqueued, asynchronous on `hip_stream`, nothing allocated, bf16
 * as uint16 storage, sparse_ffn_last_error() for the detail.
 */
#ifndef SPARSE_FFN_NORM_H
#define SPARSE_FFN_NORM_H

#include "sparse_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A [T, d] view: element (t, i) lies at data + t stride + i (stride in elements,
 * >= 0; outputs: >= d; any alignment of whole elements). */
typedef struct {
    void* data;             /* device; const where the view is an input */
    int64_t stride;
} sffn_rows_t;

typedef enum {
    SFFN_NORM_SAME = 0,     /* y in the input's type                                     */
    SFFN_NORM_INT8 = 1,     /* y int8, |entry| <= 127, and a scale for each row          */
    SFFN_NORM_E4M3 = 2      /* y 8-bit floating point (4 bits of exponent, 3 of mantissa,
                               largest 448, no infinities), and a scale for each row     */
} sffn_norm_out_t;

/* 1 <= d <= 2^20; eps positive and finite. */
typedef struct {
    int32_t d;
    sffn_dtype_t dtype;     /* of x, residual, weight, h, their gradients and y of SFFN_NORM_SAME */
    sffn_norm_out_t out;    /* forward only */
    float eps;
} sffn_norm_config_t;

/* For every row t (fp32 inside):
 *   h = x + residual, rounded to dtype (without a residual h = x)
 *   r = rsqrt(mean(h^2) + eps),   n = h w     (r = 0 where the sum of squares passes fp32)
 *   SFFN_NORM_SAME:  y = n r, rounded to dtype
 *   8 bits:          s = max|n| / 127 (or / 448), y = n / s rounded to the nearest
 *                    entry, ties to even, scale = s r; the value is y scale. The row's
 *                    factor r divides out of the entries, so that they follow from h
 *                    and w alone. A row of zeros has scale 0; one with a NaN or an infinity
 *                    in h or in h w has scale NaN and undefined entries. SFFN_NORM_SAME:
 *                    a NaN of h makes the row's y NaN, an infinity of h its own entry NaN
 *                    and the others 0; what is not finite in w shows in its own entry.
 *   x, residual (NULL: none), weight [d] (NULL: ones), y [T, d]
 *   scale [T] fp32, 8 bits only
 *   h     the sum, [T, d] or NULL; not without a residual
 * h, and with SFFN_NORM_SAME y, may be x or residual themselves (same data and stride), but
 * not each other. No output may overlap anything else. T == 0 enqueues nothing. */
sffn_status_t add_rms_norm(const sffn_norm_config_t* cfg, int64_t T, const sffn_rows_t* x,
                           const sffn_rows_t* residual, const void* weight, const sffn_rows_t* y, float* scale,
                           const sffn_rows_t* h, void* hip_stream);

/* Workspace bytes of add_rms_norm_backward where g_weight is wanted (0 when the config
 * is invalid or T <= 0). */
size_t add_rms_norm_backward_workspace_size(const sffn_norm_config_t* cfg, int64_t T);

/* Gradients of L for the gradients g_y of y and g_h of h (NULL: zero):
 *   u = g_y w,  xh = h r,  g_x = r (u - xh mean(u xh)) + g_h,  g_weight = sum_t g_y xh
 * with h the forward's sum. g_x [T, d] (dtype) is the gradient of x and of the residual
 * alike and may be h, g_y or g_h themselves (same data and stride). weight NULL: ones.
 * g_weight [d] fp32 is summed over rows in a fixed order (NULL: not wanted; zeros for
 * T == 0); it needs the workspace (256-byte aligned). */
sffn_status_t add_rms_norm_backward(const sffn_norm_config_t* cfg, int64_t T, const sffn_rows_t* h,
                                    const sffn_rows_t* g_y, const sffn_rows_t* g_h, const void* weight,
                                    const sffn_rows_t* g_x, float* g_weight, void* workspace, size_t ws_bytes,
                                    void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_FFN_NORM_H */
