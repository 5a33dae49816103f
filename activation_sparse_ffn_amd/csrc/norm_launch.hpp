// Host-side launchers of the norm with the residual's addition. Each returns the
// hipGetLastError() of its launches; callers have validated every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch.hpp"

namespace sffn {

// A [T, d] view (stride in elements).
struct Rows {
    void* p;
    int64_t stride;
};

enum class NormOut { Same = 0, Int8 = 1, E4m3 = 2 };

struct NormArgs {
    Dt dt;
    NormOut out;
    int d;
    float eps;
    int64_t T;
    Rows x, r, h, y;            // forward: r and h may be null
    Rows g_y, g_h, g_x;         // backward (x: the forward's sum); g_h may be null
    const void* w;              // [d] or null (ones)
    float* scale;               // forward in 8 bits: [T]
    float* g_w;                 // backward: [d] or null
    float* partial;             // backward with g_w: norm_partial_rows(a) rows of d
    int64_t first;              // row of the launch's first workgroup
};

int64_t norm_partial_rows(const NormArgs& a);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s);

}  // namespace sffn
