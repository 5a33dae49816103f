// The paged 8-bit cache: append of new keys and values, and the read back.
//
// A page holds P tokens of every head; keys lie [P][D], values [D][P], int8,
// with one fp32 scale for each page and head. An append of tokens x to a page
// whose first `held` tokens are of the sequence already:
//   s' = max(s, max|x| / 127) (held > 0) or max|x| / 127,
//   q' = rint(q (s / s')) for the held entries, rint(x / s') for the new ones,
// in IEEE fp32 (divisions included), so the entries are the same wherever they
// are computed.
//
// Memory-bound and small: a workgroup takes one page of one head, of keys or
// of values, so that the maximum, the rescaling and the store are one kernel
// and no two workgroups share a scale. The new values pass through LDS to be
// turned into token order; held entries are touched only where the scale grew.
#include "attn_launch.hpp"
#include "common.hpp"

namespace sffn {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPage = 128, kMaxDim = 256;

// What one workgroup works on: the call's tokens that lie in one page.
struct PageJob {
    int64_t row;        // (page id * Hkv + head): index of the scale
    int64_t t0;         // first token of the call in this page
    int held, m;        // tokens before it in the page, new tokens in the page
    int64_t early;      // call tokens before position 0 (more tokens than kv_lens says), first page's job only
    int h;
    bool values;
    bool known;         // the page is one of the pool (row is then valid)
};

// Fills the job of this workgroup; false if it has nothing to do.
__device__ bool page_job(const CacheArgs& c, int per_seq, PageJob& j) {
    int64_t id = blockIdx.x;
    j.values = id & 1;
    id >>= 1;
    j.h = (int)(id % c.Hkv);
    id /= c.Hkv;
    const int b = (int)(id / per_seq), nth = (int)(id % per_seq);
    int64_t first = b, last = b + 1;
    if (c.cu) {
        first = c.cu[b];
        last = c.cu[b + 1];
    }
    if (first < 0 || last > c.T || last <= first) return false;
    const int64_t L = c.lens[b] > 0 ? c.lens[b] : 0;
    const int64_t start = L - (last - first);                    // position of token `first`
    const int64_t from = start > 0 ? start : 0;
    const int64_t page = (from >> c.shift) + nth;
    const int64_t lo = page * c.P > from ? page * c.P : from;
    const int64_t hi = (page + 1) * c.P < L ? (page + 1) * c.P : L;
    j.early = nth == 0 && start < 0 ? -start : 0;
    j.t0 = first + (lo - start);
    j.held = (int)(lo - page * c.P);
    j.m = lo < hi ? (int)(hi - lo) : 0;
    if (j.m == 0 && j.early == 0) return false;
    int32_t pid = -1;
    if (j.m > 0 && page < c.max_pages) pid = c.table[(int64_t)b * c.table_stride + page];
    j.known = pid >= 0 && pid < c.n_pages;
    j.row = j.known ? (int64_t)pid * c.Hkv + j.h : 0;
    return true;
}

__device__ __forceinline__ int8_t requantise(int8_t q, float ratio) {
    return (int8_t)(int)rintf((float)q * ratio);
}

template <typename E>
__global__ __launch_bounds__(kThreads) void k_cache_append(const CacheArgs c, const Heads k, const Heads v,
                                                           int per_seq) {
    __shared__ uint32_t wave_max[kThreads / 64];
    __shared__ __align__(16) int8_t tile[kMaxPage * kMaxDim];   // values: new entries [token][D]
    PageJob j;
    if (!page_job(c, per_seq, j) || !j.known) return;
    const Heads& in = j.values ? v : k;
    const E* x = static_cast<const E*>(in.p) + (j.t0 * in.st + (int64_t)j.h * in.sh);
    const int chunks = c.D / 8, n = j.m * chunks;

    // max |x| as bits: larger finite values have larger bits, and infinities
    // and NaN the largest
    uint32_t most = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        float e[8];
        Elem<E>::load8(x + (int64_t)(i / chunks) * in.st + 8 * (i % chunks), e);
#pragma unroll
        for (int q = 0; q < 8; ++q) most = max(most, __float_as_uint(e[q]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) most = max(most, (uint32_t)__shfl_xor((int)most, o, 64));
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = most;
    float* scale = (j.values ? c.v_scale : c.k_scale) + j.row;
    const float old = *scale;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) most = max(most, wave_max[w]);

    float s = most >= 0x7f800000u ? __builtin_nanf("") : __uint_as_float(most) / 127.0f;
    float ratio = 1.f;
    if (j.held > 0) {
        if (!(s <= old)) {
            // the scale grows (or becomes NaN); a NaN scale stays
            if (old == old) ratio = s > 0.f ? old / s : 1.f;
            else s = old;
        } else {
            s = old;
        }
    }
    // (the barrier above is behind every thread's read of the old scale)
    if (threadIdx.x == 0) *scale = s;
    const bool regrown = ratio < 1.f;

    int8_t* pool = (j.values ? c.values : c.keys) + j.row * c.P * c.D;
    if (!j.values && regrown)
        for (int i = threadIdx.x; i < j.held * (c.D / 16); i += kThreads) {
            union { uint4 w; int8_t b[16]; } u;
            u.w = *reinterpret_cast<const uint4*>(pool + 16 * (int64_t)i);
#pragma unroll
            for (int q = 0; q < 16; ++q) u.b[q] = requantise(u.b[q], ratio);
            *reinterpret_cast<uint4*>(pool + 16 * (int64_t)i) = u.w;
        }
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int tok = i / chunks, d = 8 * (i % chunks);
        float e[8];
        Elem<E>::load8(x + (int64_t)tok * in.st + d, e);
        union { uint2 w; int8_t b[8]; } u;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            // s == 0: a maximum so small that its scale rounds to zero
            const float r = s > 0.f ? rintf(e[q] / s) : 0.f;
            u.b[q] = (int8_t)(int)fminf(fmaxf(r, -127.f), 127.f);
        }
        if (!j.values) *reinterpret_cast<uint2*>(pool + (int64_t)(j.held + tok) * c.D + d) = u.w;
        else *reinterpret_cast<uint2*>(tile + tok * c.D + d) = u.w;
    }
    if (!j.values) return;
    __syncthreads();
    // rows [D][P]: 16-token pieces that hold new tokens, or held ones to be
    // rescaled; a piece's other bytes keep what they hold
    const int end = j.held + j.m;
    const int p0 = regrown ? 0 : j.held / 16, p1 = (end + 15) / 16, np = p1 - p0;
    for (int i = threadIdx.x; i < np * c.D; i += kThreads) {
        const int d = i / np, t0 = 16 * (p0 + i % np);
        int8_t* to = pool + (int64_t)d * c.P + t0;
        union { uint4 w; int8_t b[16]; } u;
        u.w = make_uint4(0, 0, 0, 0);
        if (t0 < j.held || t0 + 16 > end) u.w = *reinterpret_cast<const uint4*>(to);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int tok = t0 + q - j.held;
            if (tok < 0) {
                if (regrown) u.b[q] = requantise(u.b[q], ratio);
            } else if (tok < j.m) {
                u.b[q] = tile[tok * c.D + d];
            }
        }
        *reinterpret_cast<uint4*>(to) = u.w;
    }
}

template <typename E> struct Store8;
template <> struct Store8<uint16_t> {
    static __device__ __forceinline__ void put(uint16_t* p, const float* v) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                  pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
};
template <> struct Store8<float> {
    static __device__ __forceinline__ void put(float* p, const float* v) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
};

template <typename E>
__global__ __launch_bounds__(kThreads) void k_cache_read(const CacheArgs c, const Heads k, const Heads v,
                                                         int per_seq) {
    // values: the page's pieces [D][P]; 16 bytes more a row than the longest
    // page, so that a column's bytes lie in other banks
    __shared__ __align__(16) int8_t tile[kMaxDim * (kMaxPage + 16)];
    PageJob j;
    if (!page_job(c, per_seq, j)) return;
    const Heads& out = j.values ? v : k;
    E* y = static_cast<E*>(out.p) + (j.t0 * out.st + (int64_t)j.h * out.sh);
    const int chunks = c.D / 8;
    const float none[8] = {__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""),
                           __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
    for (int64_t i = threadIdx.x; i < j.early * chunks; i += kThreads)
        Store8<E>::put(y + (i / chunks - j.early) * out.st + 8 * (i % chunks), none);
    if (!j.known) {
        for (int i = threadIdx.x; i < j.m * chunks; i += kThreads)
            Store8<E>::put(y + (int64_t)(i / chunks) * out.st + 8 * (i % chunks), none);
        return;
    }
    const float s = (j.values ? c.v_scale : c.k_scale)[j.row];
    const int8_t* pool = (j.values ? c.values : c.keys) + j.row * c.P * c.D;
    const int pitch = c.P + 16;
    if (j.values) {
        const int p0 = j.held / 16, np = (j.held + j.m + 15) / 16 - p0;
        for (int i = threadIdx.x; i < np * c.D; i += kThreads) {
            const int d = i / np, t0 = 16 * (p0 + i % np);
            *reinterpret_cast<uint4*>(tile + d * pitch + t0) =
                *reinterpret_cast<const uint4*>(pool + (int64_t)d * c.P + t0);
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < j.m * chunks; i += kThreads) {
        const int tok = i / chunks, d = 8 * (i % chunks);
        union { uint2 w; int8_t b[8]; } u;
        if (j.values) {
#pragma unroll
            for (int q = 0; q < 8; ++q) u.b[q] = tile[(d + q) * pitch + j.held + tok];
        } else {
            u.w = *reinterpret_cast<const uint2*>(pool + (int64_t)(j.held + tok) * c.D + d);
        }
        float e[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) e[q] = (float)u.b[q] * s;
        Store8<E>::put(y + (int64_t)tok * out.st + d, e);
    }
}

}  // namespace

hipError_t launch_cache_append(const CacheArgs& c, const Heads& k, const Heads& v, hipStream_t s) {
    const int per_seq = (int)pages_touched(c.max_new, c.P);
    const dim3 grid((unsigned)cache_copy_blocks(c));
    if (c.dt == Dt::BF16) k_cache_append<uint16_t><<<grid, kThreads, 0, s>>>(c, k, v, per_seq);
    else k_cache_append<float><<<grid, kThreads, 0, s>>>(c, k, v, per_seq);
    return hipGetLastError();
}

hipError_t launch_cache_read(const CacheArgs& c, const Heads& k, const Heads& v, hipStream_t s) {
    const int per_seq = (int)pages_touched(c.max_new, c.P);
    const dim3 grid((unsigned)cache_copy_blocks(c));
    if (c.dt == Dt::BF16) k_cache_read<uint16_t><<<grid, kThreads, 0, s>>>(c, k, v, per_seq);
    else k_cache_read<float><<<grid, kThreads, 0, s>>>(c, k, v, per_seq);
    return hipGetLastError();
}

}  // namespace sffn
