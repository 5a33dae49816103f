// The paged 4-bit cache: new tokens stored, tokens read back.
//
//   keys: for 32 channels e = the least power of two with max|k| <= 6 e, entry k / e;
//   values: s = max|v| / 6 of the token and head, entry v / s;
//   entries rounded to {0, 0.5, 1, 1.5, 2, 3, 4, 6}, ties to the even code.
//
// A lane has eight channels of a token and head, keys and values alike: 16 bytes in (fp32:
// two times 16), 4 bytes of entries out. Largest values are compared as integers, in which
// infinities and NaN come out on top. Every token's scales are its own: nothing that is held
// is touched, and a lane needs no more than shuffles with its neighbours.
//
// Memory-bound, and for few tokens bound by the chain of loads from offsets to table entry:
// 4096 tokens of 8 heads of 128 in 7.8 us stored and 7.1 read (21 MB in all: 2.8 TB/s; an
// empty launch and a copy of as much take 3.5 + 4.1), 32 single tokens 3.6 and 3.5. With the
// slots given an append looks up no pages; the offsets alone where a sequence of the call can
// have more than max_new tokens (32 single tokens 0.4 us of it, 32 times 128 of them 0.9).
#include "attn_common.hpp"

namespace sffn {

namespace {

constexpr int kThreads = 256;

// The sequence in which token t of the call lies, if it is in one, and its first token: the
// last of n ascending offsets that is not above t (sequence 0 if none is). Found by the L
// lanes of a row together, L offsets at a time: of 32 in two loads one after another, where
// halving takes five and one for the offset.
template <int L>
__device__ __forceinline__ int sequence_at(const int32_t* offsets, int n, int t, int& first) {
    if (n == 1) {           // nothing to search, and nothing waits for the others' offsets
        first = offsets[0];
        return 0;
    }
    const uint32_t lane = threadIdx.x % L, group = (threadIdx.x & 63) / L * L;
    uint32_t lo = 0, hi = (uint32_t)n, step;
    first = 0x7fffffff;
    do {
        step = (hi - lo + L - 1) / L;
        const uint32_t i = lo + lane * step;
        const int at = i < hi ? offsets[i] : 0x7fffffff;
        const int k = __popcll(__ballot(at <= t) >> group & (((uint64_t)1 << L) - 1));
        if (k == 0) break;
        first = __shfl(at, (int)group + k - 1, 64);
        lo += (k - 1) * step;
        hi = min(lo + step, hi);
    } while (step > 1);
    return (int)lo;
}

// Where token t of the call lies: its slot, kLost where it shows as NaN (beyond max_new,
// offsets that leave the call, no page), kNone in no sequence.
constexpr int64_t kLost = -1, kNone = -2;
template <int L>
__device__ __forceinline__ int64_t slot_of(const CacheArgs& c, int t) {
    int b = t, first = t, last = t + 1;
    if (c.cu) {
        b = sequence_at<L>(c.cu, c.B, t, first);
        last = c.cu[b + 1];
        if (t < first || t >= last) return kNone;
        if (first < 0 || last > c.T || t - first >= c.max_new) return kLost;
    }
    const int64_t pos = (int64_t)c.lens[b] - (last - first) + (t - first);
    if (pos < 0 || (pos >> c.shift) >= c.max_pages) return kLost;
    const uint32_t page = (uint32_t)c.table[(int64_t)b * c.table_stride + (pos >> c.shift)];
    if (page >= (uint64_t)c.n_pages) return kLost;
    return ((int64_t)page << c.shift) + (pos & (c.P - 1));
}

// The slot that the caller gives it, unless the batch's offsets (where they count, see
// kv_cache4_append) have it beyond max_new.
template <int L>
__device__ __forceinline__ int64_t slot_given(const CacheArgs& c, const int64_t* slots, int t) {
    const int64_t slot = slots[t];
    if (!c.cu) return slot;
    int first;
    sequence_at<L>(c.cu, c.B, t, first);
    return (int64_t)t - first >= c.max_new ? kLost : slot;
}

// Row (token of a page and head) of the cache's arrays.
__device__ __forceinline__ int64_t row_of_slot(const CacheArgs& c, int64_t slot, int h) {
    return (((slot >> c.shift) * c.Hkv + h) << c.shift) + (slot & (c.P - 1));
}

// Eight entries of x, already divided by their scale but for the power of two `by`.
__device__ __forceinline__ uint32_t entries8(const float* x, float by) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], by, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], by, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], by, 2);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], by, 3);
}
__device__ __forceinline__ void values8(uint32_t w, float* x) {
#define SFFN_TWO(i)                                                                   \
    {                                                                                 \
        const auto p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, i);           \
        x[2 * i] = p[0];                                                              \
        x[2 * i + 1] = p[1];                                                          \
    }
    SFFN_TWO(0) SFFN_TWO(1) SFFN_TWO(2) SFFN_TWO(3)
#undef SFFN_TWO
}

// Largest magnitude of eight, as an integer (NaN above infinity above numbers), over
// groups of LANES lanes.
template <int LANES>
__device__ __forceinline__ uint32_t largest(const float* x) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
    return m;
}

// Rows (token, head) that a workgroup takes at a time.
constexpr int rows_each(int D) { return kThreads * 8 / D; }

template <typename E, int D>
__global__ __launch_bounds__(kThreads) void k_cache4_append(const CacheArgs c, const Cache4 cache, const int64_t* slots,
                                                            const Heads k, const Heads v, uint32_t first) {
    const uint32_t r = (first + blockIdx.x) * rows_each(D) + threadIdx.x / (D / 8);     // of fewer than 2^31
    if (r >= (uint32_t)(c.T * c.Hkv)) return;       // whole groups of D / 8 lanes
    const int t = (int)(r / (uint32_t)c.Hkv), h = (int)(r - (uint32_t)t * (uint32_t)c.Hkv);
    const int d = threadIdx.x % (D / 8) * 8;
    float x[8], y[8];
    Elem<E>::load8(static_cast<const E*>(k.p) + (t * k.st + h * k.sh) + d, x);
    Elem<E>::load8(static_cast<const E*>(v.p) + (t * v.st + h * v.sh) + d, y);
    const int64_t slot = slots ? slot_given<D / 8>(c, slots, t) : slot_of<D / 8>(c, t);
    const bool stored = slot >= 0 && slot < c.n_pages << c.shift;
    const int64_t row = row_of_slot(c, stored ? slot : 0, h);

    const uint32_t top = largest<4>(x);     // of 32 channels
    int e = max((int)(top >> 23) - 2 + ((top & 0x7fffffu) > 0x400000u), 0);
    if (top >= 0x7f800000u) e = 255;
    // powers of two below fp32's normal numbers: both sides 2^64 larger
    const bool low = e < 64;
    if (low)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= 0x1p64f;
    const uint32_t kw = entries8(x, __uint_as_float((uint32_t)(low ? e + 64 : e == 255 ? 127 : e) << 23));

    const uint32_t most = largest<D / 8>(y);        // of the head
    const float s = most >= 0x7f800000u ? __builtin_nanf("") : __uint_as_float(most) / 6.f;
    // y / s as IEEE division rounds it: with the rounded 1 / s one correction of y times that
    // does it (P. Markstein), while nothing on the way is subnormal; what is then below 2^-24
    // of s is entry 0 in any case. (8 divisions a lane and 64-bit row numbers: 8.7 us
    // for the 4096 tokens above.)
    const float up = s < 0x1p-60f ? 0x1p64f : 1.f, su = s * up, inv = 1.f / su;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float yu = y[i] * up, q = yu * inv;
        y[i] = s > 0.f ? __builtin_fmaf(__builtin_fmaf(-q, su, yu), inv, q) : 0.f;
    }
    const uint32_t vw = entries8(y, 1.f);
    if (!stored) return;
    *reinterpret_cast<uint32_t*>(cache.keys + row * (D / 2) + d / 2) = kw;
    *reinterpret_cast<uint32_t*>(cache.values + row * (D / 2) + d / 2) = vw;
    if (d % 32 == 0) cache.k_exp[row * (D / 32) + d / 32] = (uint8_t)e;
    if (d == 0) cache.v_scale[row] = s;
}

template <typename E, int D>
__global__ __launch_bounds__(kThreads) void k_cache4_read(const CacheArgs c, const Cache4 cache, const Heads k,
                                                          const Heads v, uint32_t first) {
    const uint32_t r = (first + blockIdx.x) * rows_each(D) + threadIdx.x / (D / 8);
    if (r >= (uint32_t)(c.T * c.Hkv)) return;
    const int t = (int)(r / (uint32_t)c.Hkv), h = (int)(r - (uint32_t)t * (uint32_t)c.Hkv);
    const int d = threadIdx.x % (D / 8) * 8;
    const int64_t slot = slot_of<D / 8>(c, t);
    if (slot == kNone) return;
    float x[8], y[8];
    if (slot == kLost) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = y[i] = __builtin_nanf("");
    } else {
        const int64_t row = row_of_slot(c, slot, h);
        const uint32_t kw = *reinterpret_cast<const uint32_t*>(cache.keys + row * (D / 2) + d / 2);
        const uint32_t vw = *reinterpret_cast<const uint32_t*>(cache.values + row * (D / 2) + d / 2);
        const int e = cache.k_exp[row * (D / 32) + d / 32];
        const float s = cache.v_scale[row];
        values8(kw, x);
        values8(vw, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[i] = e == 255 ? __builtin_nanf("") : ldexpf(x[i], e - 127);
            y[i] *= s;
        }
    }
    store8(static_cast<E*>(k.p) + (t * k.st + h * k.sh) + d, x);
    store8(static_cast<E*>(v.p) + (t * v.st + h * v.sh) + d, y);
}

template <typename E, int D>
hipError_t append(const CacheArgs& c, const Cache4& b, const int64_t* slots, const Heads& k, const Heads& v,
                  hipStream_t s) {
    return launch_in_pieces((c.T * c.Hkv + rows_each(D) - 1) / rows_each(D), [&](uint32_t first, unsigned n) {
        k_cache4_append<E, D><<<dim3(n), kThreads, 0, s>>>(c, b, slots, k, v, first);
    });
}

template <typename E, int D>
hipError_t read(const CacheArgs& c, const Cache4& b, const Heads& k, const Heads& v, hipStream_t s) {
    return launch_in_pieces((c.T * c.Hkv + rows_each(D) - 1) / rows_each(D), [&](uint32_t first, unsigned n) {
        k_cache4_read<E, D><<<dim3(n), kThreads, 0, s>>>(c, b, k, v, first);
    });
}

// f(element type, head width)
template <typename F>
hipError_t by_kind(const CacheArgs& c, F f) {
    auto width = [&](auto e) {
        switch (c.D) {
            case 64: return f(e, std::integral_constant<int, 64>{});
            case 128: return f(e, std::integral_constant<int, 128>{});
            default: return f(e, std::integral_constant<int, 256>{});
        }
    };
    return c.dt == Dt::BF16 ? width((uint16_t)0) : width(0.f);
}

}  // namespace

hipError_t launch_cache4_append(const CacheArgs& c, const Cache4& b, const int64_t* slots, const Heads& k,
                                const Heads& v, hipStream_t s) {
    return by_kind(c, [&](auto e, auto d) { return append<decltype(e), d.value>(c, b, slots, k, v, s); });
}

hipError_t launch_cache4_read(const CacheArgs& c, const Cache4& b, const Heads& k, const Heads& v, hipStream_t s) {
    return by_kind(c, [&](auto e, auto d) { return read<decltype(e), d.value>(c, b, k, v, s); });
}

}  // namespace sffn
