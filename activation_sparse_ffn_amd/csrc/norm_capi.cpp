// C ABI of the norm with the residual's addition (include/sparse_ffn_norm.h): argument
// checks, workspace sizes and the calls of the launchers.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/sparse_ffn_norm.h"
#include "norm_launch.hpp"
#include "status.hpp"

namespace {

using sffn::as_int;
using sffn::fail;
using sffn::hip_status;

// Bounds that keep every size product below 2^63.
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int32_t kMaxWidth = 1 << 20;
constexpr int64_t kMaxStride = (int64_t)1 << 31;

#define SFFN_TRY(call)                        \
    do {                                      \
        const sffn_status_t try_st = (call);  \
        if (try_st != SFFN_OK) return try_st; \
    } while (0)

sffn_status_t check_config(const sffn_norm_config_t* c, int64_t T) {
    if (!c) return fail(SFFN_ERR_INVALID_ARG, "config is null");
    if (c->d < 1 || c->d > kMaxWidth)
        return fail(SFFN_ERR_INVALID_ARG, "d must lie in [1, 2^20] (got %d)", c->d);
    const int dtype = as_int(c->dtype), out = as_int(c->out);
    if (dtype != SFFN_F32 && dtype != SFFN_BF16) return fail(SFFN_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (out != SFFN_NORM_SAME && out != SFFN_NORM_INT8 && out != SFFN_NORM_E4M3)
        return fail(SFFN_ERR_INVALID_ARG, "unknown output %d", out);
    if (!(c->eps > 0.f && std::isfinite(c->eps)))
        return fail(SFFN_ERR_INVALID_ARG, "eps must be positive and finite (got %g)", (double)c->eps);
    if (T < 0) return fail(SFFN_ERR_INVALID_ARG, "T must be >= 0 (got %lld)", (long long)T);
    if (T > kMaxRows) return fail(SFFN_ERR_UNSUPPORTED, "T = %lld is too large for one call", (long long)T);
    return SFFN_OK;
}

size_t elem_size(const sffn_norm_config_t* c) { return as_int(c->dtype) == SFFN_BF16 ? 2 : 4; }

sffn_status_t check_rows(const sffn_rows_t* v, const char* name, const sffn_norm_config_t* c, int64_t T, size_t e,
                         bool out) {
    if (!v || !v->data) return fail(SFFN_ERR_INVALID_ARG, "%s is null", name);
    if (v->stride < 0 || v->stride > kMaxStride)
        return fail(SFFN_ERR_INVALID_ARG, "%s has a stride out of range (%lld)", name, (long long)v->stride);
    if (reinterpret_cast<uintptr_t>(v->data) % e != 0)
        return fail(SFFN_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
    if (out && T > 1 && v->stride < c->d) return fail(SFFN_ERR_INVALID_ARG, "%s overlaps itself", name);
    return SFFN_OK;
}

// An output that lies where an input does must write every row over itself: over another
// one it would meet a workgroup that has yet to read it.
sffn_status_t check_in_place(const sffn_rows_t* out, const char* name, const sffn_rows_t* in, const char* input, int64_t T,
                             bool same_size = true) {
    if (!in || out->data != in->data || (same_size && (T == 1 || out->stride == in->stride))) return SFFN_OK;
    return fail(SFFN_ERR_INVALID_ARG, "%s lies where %s does, with rows of another size", name, input);
}

sffn_status_t check_vector(const void* p, const char* name, size_t e) {
    if (reinterpret_cast<uintptr_t>(p) % e != 0)
        return fail(SFFN_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
    return SFFN_OK;
}

sffn::Rows view(const sffn_rows_t* v) { return v ? sffn::Rows{v->data, v->stride} : sffn::Rows{nullptr, 0}; }

sffn::NormArgs norm_args(const sffn_norm_config_t* c, int64_t T, const void* weight) {
    sffn::NormArgs a{};
    a.dt = as_int(c->dtype) == SFFN_BF16 ? sffn::Dt::BF16 : sffn::Dt::F32;
    a.out = static_cast<sffn::NormOut>(as_int(c->out));
    a.d = c->d;
    a.eps = c->eps;
    a.T = T;
    a.w = weight;
    return a;
}

size_t partial_bytes(const sffn::NormArgs& a) { return (size_t)sffn::norm_partial_rows(a) * a.d * 4; }

}  // namespace

extern "C" {

sffn_status_t add_rms_norm(const sffn_norm_config_t* cfg, int64_t T, const sffn_rows_t* x,
                           const sffn_rows_t* residual, const void* weight, const sffn_rows_t* y, float* scale,
                           const sffn_rows_t* h, void* hip_stream) {
    SFFN_TRY(check_config(cfg, T));
    if (T == 0) return SFFN_OK;
    const size_t e = elem_size(cfg);
    const bool wide = as_int(cfg->out) != SFFN_NORM_SAME;
    SFFN_TRY(check_rows(x, "x", cfg, T, e, false));
    if (residual) SFFN_TRY(check_rows(residual, "residual", cfg, T, e, false));
    SFFN_TRY(check_vector(weight, "weight", e));
    SFFN_TRY(check_rows(y, "y", cfg, T, wide ? 1 : e, true));
    SFFN_TRY(check_in_place(y, "y", x, "x", T, !wide));
    SFFN_TRY(check_in_place(y, "y", residual, "residual", T, !wide));
    if (wide && !scale) return fail(SFFN_ERR_INVALID_ARG, "scale is null");
    SFFN_TRY(check_vector(scale, "scale", 4));
    if (h) {
        if (!residual) return fail(SFFN_ERR_INVALID_ARG, "h is the sum with the residual, which is not given");
        SFFN_TRY(check_rows(h, "h", cfg, T, e, true));
        SFFN_TRY(check_in_place(h, "h", x, "x", T));
        SFFN_TRY(check_in_place(h, "h", residual, "residual", T));
        if (h->data == y->data) return fail(SFFN_ERR_INVALID_ARG, "h and y are the same");
    }
    sffn::NormArgs a = norm_args(cfg, T, weight);
    a.x = view(x);
    a.r = view(residual);
    a.y = view(y);
    a.h = view(h);
    a.scale = scale;
    return hip_status(sffn::launch_norm(a, static_cast<hipStream_t>(hip_stream)), "add_rms_norm");
}

size_t add_rms_norm_backward_workspace_size(const sffn_norm_config_t* cfg, int64_t T) {
    if (check_config(cfg, T) != SFFN_OK || T == 0) return 0;
    return partial_bytes(norm_args(cfg, T, nullptr));
}

sffn_status_t add_rms_norm_backward(const sffn_norm_config_t* cfg, int64_t T, const sffn_rows_t* h,
                                    const sffn_rows_t* g_y, const sffn_rows_t* g_h, const void* weight,
                                    const sffn_rows_t* g_x, float* g_weight, void* workspace, size_t ws_bytes,
                                    void* hip_stream) {
    SFFN_TRY(check_config(cfg, T));
    SFFN_TRY(check_vector(g_weight, "g_weight", 4));
    hipStream_t s = static_cast<hipStream_t>(hip_stream);
    if (T == 0)
        return hip_status(g_weight ? sffn::launch_zero_f32(g_weight, cfg->d, s) : hipSuccess, "add_rms_norm_backward");
    const size_t e = elem_size(cfg);
    SFFN_TRY(check_rows(h, "h", cfg, T, e, false));
    SFFN_TRY(check_rows(g_y, "g_y", cfg, T, e, false));
    if (g_h) SFFN_TRY(check_rows(g_h, "g_h", cfg, T, e, false));
    SFFN_TRY(check_vector(weight, "weight", e));
    SFFN_TRY(check_rows(g_x, "g_x", cfg, T, e, true));
    SFFN_TRY(check_in_place(g_x, "g_x", h, "h", T));
    SFFN_TRY(check_in_place(g_x, "g_x", g_y, "g_y", T));
    SFFN_TRY(check_in_place(g_x, "g_x", g_h, "g_h", T));
    sffn::NormArgs a = norm_args(cfg, T, weight);
    a.x = view(h);
    a.g_y = view(g_y);
    a.g_h = view(g_h);
    a.g_x = view(g_x);
    if (g_weight) {
        const size_t need = partial_bytes(a);
        if (!workspace) return fail(SFFN_ERR_INVALID_ARG, "workspace is null");
        if ((reinterpret_cast<uintptr_t>(workspace) & 255) != 0)
            return fail(SFFN_ERR_INVALID_ARG, "workspace is not 256-byte aligned");
        if (ws_bytes < need)
            return fail(SFFN_ERR_WORKSPACE, "workspace holds %zu bytes, %zu needed", ws_bytes, need);
        a.g_w = g_weight;
        a.partial = static_cast<float*>(workspace);
    }
    return hip_status(sffn::launch_norm_backward(a, s), "add_rms_norm_backward");
}

}  // extern "C"
