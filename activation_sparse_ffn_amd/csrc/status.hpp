// What the C entry points share: the last failure's detail and small checks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "../../include/sparse_ffn.h"

namespace sffn {

// Detail of the last failure on the calling thread: a fixed array, so that no
// entry point can throw while it reports.
inline thread_local char last_error[512];

inline sffn_status_t fail(sffn_status_t st, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(last_error, sizeof last_error, fmt, ap);
    va_end(ap);
    return st;
}

inline sffn_status_t hip_status(hipError_t e, const char* what) {
    if (e == hipSuccess) return SFFN_OK;
    return fail(SFFN_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The enum fields come from C callers as plain ints: they are read as ints (an
// out-of-range value read as a C++ enum is undefined behaviour).
template <typename Enum>
int as_int(const Enum& e) {
    static_assert(sizeof(Enum) == sizeof(int), "enums of the C ABI are int-sized");
    int v;
    std::memcpy(&v, &e, sizeof v);
    return v;
}

}  // namespace sffn
