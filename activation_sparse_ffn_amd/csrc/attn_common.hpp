// Device helpers that the attention-side kernels share.
#pragma once

#include "attn_launch.hpp"
#include "common.hpp"

namespace sffn {

// Tokens [from, to) of the call that belong to sequence b and are not computed: those
// beyond its first max_new, or all of a sequence whose offsets leave the call. Their
// rows are made NaN. False if there are none.
__device__ __forceinline__ bool lost_tokens(const CacheArgs& c, int b, int& from, int& to) {
    if (!c.cu) return false;            // one token each
    const int T = (int)c.T, first = c.cu[b], last = c.cu[b + 1];
    const bool inside = first >= 0 && last <= T;
    from = inside ? first + c.max_new : first > 0 ? first : 0;
    to = last < T ? last : T;
    return from < to;
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two fp32 rounded to bf16, to nearest even, as one word (one instruction).
__device__ __forceinline__ uint32_t round2(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x, y}), bf16x2));
}

__device__ __forceinline__ void store4(uint16_t* p, const float* v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(round2(v[0], v[1]), round2(v[2], v[3]));
}
__device__ __forceinline__ void store4(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float* v) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(round2(v[0], v[1]), round2(v[2], v[3]), round2(v[4], v[5]), round2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

}  // namespace sffn
