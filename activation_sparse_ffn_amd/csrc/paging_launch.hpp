// Host-side launchers of the page bookkeeping. Each returns the hipGetLastError() of its
// launches; callers have validated every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch.hpp"

namespace sffn {

// Positions and slots of the tokens of a batch.
struct SlotArgs {
    const int32_t* table;           // [B] rows of max_pages
    int64_t table_stride;
    const int32_t* lens;            // [B], new tokens included
    const int32_t* cu;              // [B + 1] or null (token b belongs to sequence b)
    int B, max_pages, max_new, shift;
    int64_t n_pages, T;
    int32_t* positions;
    int64_t* slots;
};
hipError_t launch_slots(const SlotArgs& a, hipStream_t s);

struct PlanArgs {
    int32_t* table;
    int64_t table_stride;
    int32_t* free_pages;
    int64_t n_pages, T;
    int B, max_pages, shift;
    const int32_t *lens, *keep, *fresh, *n_free;    // keep may be null
    int32_t *lens_out, *n_free_out, *cu, *positions;
    int64_t* slots;
};
hipError_t launch_page_plan(const PlanArgs& a, hipStream_t s);

}  // namespace sffn
