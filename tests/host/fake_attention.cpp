// A stand-in for the HIP runtime and for the launchers of the attention-side
// operators, so that their C entry points' host logic can be built with the
// sanitizers and run without a GPU. Every launch records itself and returns the
// status the test asks for.
#include <cstdint>

#include <hip/hip_runtime_api.h>

#include "attn_launch.hpp"

hipError_t g_fake_launch_status = hipSuccess;
int g_fake_launches = 0;
sffn::AttnPlan g_fake_plan{};

extern "C" {
const char* hipGetErrorString(hipError_t e) { return e == hipSuccess ? "no error" : "injected HIP error"; }
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 256; return hipSuccess; }
}

namespace sffn {
static hipError_t launched() {
    ++g_fake_launches;
    return g_fake_launch_status;
}
size_t rope_partial_floats(const RopeArgs& a) { return a.norm ? (size_t)1024 * 2 * a.D : 0; }
hipError_t launch_rope(const RopeArgs&, hipStream_t) { return launched(); }
hipError_t launch_rope_backward(const RopeArgs&, hipStream_t) { return launched(); }
hipError_t launch_cache_append(const CacheArgs&, const Heads&, const Heads&, hipStream_t) { return launched(); }
hipError_t launch_cache_read(const CacheArgs&, const Heads&, const Heads&, hipStream_t) { return launched(); }
hipError_t launch_cache_attention(const CacheArgs&, const AttnPlan& plan, const Heads&, int, float, int, const Heads&,
                                  float*, void*, hipStream_t) {
    g_fake_plan = plan;
    return launched();
}
hipError_t launch_zero_f32(float*, int64_t, hipStream_t) { return launched(); }
}  // namespace sffn
