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
// and no two workgroups share a scale; what it costs is the chain lengths ->
// table -> rows -> maximum -> store, so a thread's loads are all in flight at once
// and stay in registers for the rounding. (In an append the link from the table to
// the rows is the code's own: page_job reads the entry first, though the new tokens'
// addresses do not need it. In a read it is the data's.) A thread's piece is four tokens of
// eight channels: four tokens of a channel are one word of the values' order
// ([D][P]), which they reach through LDS in whole words. Held entries are touched
// only where the scale grew.
//
// One token in each of 32 sequences (8 heads of 128): 5.7 us, launch and chain (fp32
// 5.7; 7.6 where every scale grows and up to 63 held tokens are rounded again). A chunk of 4095 tokens (17 MB in, 8.4 MB out, a copy's 5 us): 12.2 us, one
// round of 1040 workgroups that all wait for the same links of the chain; with the
// values' bytes stored one at a time 16.7; from fp32 12.1. Reading that chunk back:
// 7.8 us, 3.2 TB/s, to fp32 12.4.
#include "attn_common.hpp"
#include "attn_launch.hpp"

namespace sffn {

namespace {

constexpr int kThreads = 256;

// What one workgroup works on: the call's tokens that lie in one page.
struct PageJob {
    int64_t row;        // (page id * Hkv + head): index of the scale
    int64_t t0;         // first token of the call in this page
    int held, m;        // tokens before it in the page, new tokens in the page
    int64_t early;      // call tokens before position 0 (more tokens than kv_lens says), first page's job only
    bool beside;        // first page's job, which has the sequence's lost tokens to itself
    int b, h;
    bool values;
    bool known;         // the page is one of the pool (row is then valid)
};

// The last sequence whose places begin at `place` or before: the wave looks at 64
// sequences at a time, evenly apart and then closer.
__device__ __forceinline__ int sequence_at(const CacheArgs& c, int64_t place) {
    const int lane = threadIdx.x & 63;
    int lo = 0, hi = c.B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64, b = lane < (hi - lo + step - 1) / step ? lo + lane * step : -1;
        const int at = b >= 0 ? c.cu[b] : 0;
        const uint64_t before = __ballot(b >= 0 && first_place(at > 0 ? at : 0, b, c.shift) <= place);
        const int k = before != 0 ? __popcll(before) - 1 : 0;
        lo += k * step;
        if (hi - lo > step) hi = lo + step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// Fills the job of this workgroup; false if it has no token. per_seq: places of each
// sequence, 0 where they are by the call's tokens.
__device__ bool page_job(const CacheArgs& c, int per_seq, uint32_t first_block, PageJob& j) {
    uint32_t id = first_block + blockIdx.x;
    j.values = id & 1;
    id >>= 1;
    j.h = (int)(id % (uint32_t)c.Hkv);
    id /= (uint32_t)c.Hkv;
    int b, nth;
    j.beside = false;
    if (per_seq > 0) {
        b = (int)(id / (uint32_t)per_seq);
        nth = (int)(id % (uint32_t)per_seq);
    } else {
        b = sequence_at(c, id);
        const int at = c.cu[b];
        nth = (int)(id - first_place(at > 0 ? at : 0, b, c.shift));
        if (nth < 0) return false;          // offsets that do not begin with 0
    }
    j.b = b;
    j.beside = nth == 0;
    int64_t first = b, last = b + 1;
    if (c.cu) {
        first = c.cu[b];
        last = c.cu[b + 1];
    }
    if (first < 0 || last > c.T || last <= first) return false;
    const int64_t start = (c.lens[b] > 0 ? c.lens[b] : 0) - (last - first);     // position of token `first`
    const int64_t end = start + (last - first < c.max_new ? last - first : c.max_new);
    const int64_t from = start > 0 ? start : 0;
    const int64_t page = (from >> c.shift) + nth;
    const int64_t lo = page * c.P > from ? page * c.P : from;
    const int64_t hi = (page + 1) * c.P < end ? (page + 1) * c.P : end;
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

// rint(x / s) of eight values, |x| <= 127 s but for the rounding of s, in the low
// bytes of b. x (1 / s) + 1.5 2^23 holds the rounded quotient in its low bits; 1 /
// s is within 2^-24 of itself, so that is rint(x / s) unless the quotient lies
// within 2^-15 of a half. Where one of the eight does (or s is so small that 1 / s
// might overflow; the quotient may then pass 127 too) all eight are divided.
__device__ __forceinline__ void quantise8(const float* x, float s, float inverse, uint32_t* b) {
    const float magic = 12582912.f;
    float off = 0.f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const float y = __builtin_fmaf(x[p], inverse, magic);
        off = fmaxf(off, fabsf(__builtin_fmaf(x[p], inverse, magic - y)));
        b[p] = __float_as_uint(y);
    }
    if (off > 0.4999f || s < 1e-30f) {
#pragma unroll
        for (int p = 0; p < 8; ++p) b[p] = (uint32_t)(int)fminf(fmaxf(rintf(x[p] / s), -127.f), 127.f);
    }
}

// The low bytes of four words as one.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
    return lo | hi;
}

// LDS row pitch of the values' tile [D][P], in bytes: one word more than the
// page, so that the rows of eight channels apart lie in other banks.
__device__ __forceinline__ int tile_pitch(int P) { return P + 4; }
// It is allotted at the launch, for the cache's own sizes: with room for the
// largest page and head four workgroups would fill a compute unit, and the 65
// pages of a chunk that starts inside one (1040 workgroups) take two rounds.
inline size_t tile_bytes(const CacheArgs& c) { return (size_t)c.D * (c.P + 4); }

// The largest |x| of eight elements, as the bits of an fp32.
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t raw_most(const Raw<uint16_t>& r) {
    const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu));
    return (uint32_t)max(m.x, m.y) << 16;
}
__device__ __forceinline__ uint32_t raw_most(const Raw<float>& r) {
    const float x[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return m;
}

template <typename E>
__global__ __launch_bounds__(kThreads) void k_cache_append(const CacheArgs c, const Heads k, const Heads v,
                                                           int per_seq, uint32_t first_block) {
    __shared__ uint32_t wave_max[kThreads / 64];
    extern __shared__ uint32_t tile[];      // values: new entries, four tokens a word
    PageJob j;
    if (!page_job(c, per_seq, first_block, j) || !j.known) return;
    const Heads& in = j.values ? v : k;
    const E* x = static_cast<const E*>(in.p) + (j.t0 * in.st + (int64_t)j.h * in.sh);
    float* scale = (j.values ? c.v_scale : c.k_scale) + j.row;
    const float old = *scale;
    // piece i: slots 4 g .. 4 g + 3 of the page, channels 8 (i % chunks) ..
    const int chunks = c.D / 8, g0 = j.held / 4, n = ((j.held + j.m + 3) / 4 - g0) * chunks;
    auto load = [&](int i, Raw<E>* raw) {
        const int tok = 4 * (g0 + i / chunks) - j.held, d = 8 * (i % chunks);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (tok + q >= 0 && tok + q < j.m) raw[q].load(x + (int64_t)(tok + q) * in.st + d);
    };

    // max |x| as bits: larger finite values have larger bits, and infinities
    // and NaN the largest
    uint32_t most = 0;
    auto widest = [&](int i, const Raw<E>* raw) {
        const int tok = 4 * (g0 + i / chunks) - j.held;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (tok + q < 0 || tok + q >= j.m) continue;
            most = max(most, raw_most(raw[q]));
        }
    };
    Raw<E> first[4];        // the thread's first piece: its only one for 64 tokens of 128 channels
    if ((int)threadIdx.x < n) {
        load(threadIdx.x, first);
        widest(threadIdx.x, first);
    }
    for (int i = threadIdx.x + kThreads; i < n; i += kThreads) {
        Raw<E> raw[4];
        load(i, raw);
        widest(i, raw);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) most = max(most, (uint32_t)__shfl_xor((int)most, o, 64));
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = most;
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
    const float inverse = 1.f / s;

    int8_t* pool = (j.values ? c.values : c.keys) + j.row * c.P * c.D;
    const int pitch = tile_pitch(c.P) / 4;
    if (!j.values && regrown)
        for (int i = threadIdx.x; i < j.held * (c.D / 16); i += kThreads) {
            union { uint4 w; int8_t b[16]; } u;
            u.w = *reinterpret_cast<const uint4*>(pool + 16 * (int64_t)i);
#pragma unroll
            for (int q = 0; q < 16; ++q) u.b[q] = requantise(u.b[q], ratio);
            *reinterpret_cast<uint4*>(pool + 16 * (int64_t)i) = u.w;
        }
    auto round = [&](int i, const Raw<E>* raw) {
        const int g = g0 + i / chunks, tok = 4 * g - j.held, d = 8 * (i % chunks);
        uint32_t b[4][8] = {};  // zeros under a scale of 0 (a maximum too small for one) or NaN
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (tok + q < 0 || tok + q >= j.m) continue;
            float e[8];
            raw[q].decode(e);
            if (s > 0.f) quantise8(e, s, inverse, b[q]);
            if (!j.values)
                *reinterpret_cast<uint2*>(pool + (int64_t)(4 * g + q) * c.D + d) =
                    make_uint2(low_bytes(b[q][0], b[q][1], b[q][2], b[q][3]),
                               low_bytes(b[q][4], b[q][5], b[q][6], b[q][7]));
        }
        if (j.values)
#pragma unroll
            for (int p = 0; p < 8; ++p) tile[(d + p) * pitch + g] = low_bytes(b[0][p], b[1][p], b[2][p], b[3][p]);
    };
    if ((int)threadIdx.x < n) round(threadIdx.x, first);
    for (int i = threadIdx.x + kThreads; i < n; i += kThreads) {
        Raw<E> raw[4];
        load(i, raw);
        round(i, raw);
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
        const uint32_t* from = tile + d * pitch + t0 / 4;
        if (t0 >= j.held && t0 + 16 <= end) {
            *reinterpret_cast<uint4*>(to) = make_uint4(from[0], from[1], from[2], from[3]);
            continue;
        }
        const uint4 was = *reinterpret_cast<const uint4*>(to);
        uint32_t w[4] = {was.x, was.y, was.z, was.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int t = t0 + 4 * q;
            if (regrown && t < j.held) {
                uint32_t r = 0;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int8_t old_q = (int8_t)(w[q] >> (8 * p));
                    r |= (uint32_t)(uint8_t)(t + p < j.held ? requantise(old_q, ratio) : old_q) << (8 * p);
                }
                w[q] = r;
            }
            // bytes of the word that are new tokens
            uint32_t fresh = 0;
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (t + p >= j.held && t + p < end) fresh |= 255u << (8 * p);
            if (fresh != 0) w[q] = (w[q] & ~fresh) | (from[q] & fresh);
        }
        *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <typename E>
__global__ __launch_bounds__(kThreads) void k_cache_read(const CacheArgs c, const Heads k, const Heads v,
                                                         int per_seq, uint32_t first_block) {
    extern __shared__ uint32_t tile[];      // values: the page's rows [D][P]
    PageJob j;
    const bool any = page_job(c, per_seq, first_block, j);
    const Heads& out = j.values ? v : k;
    const int chunks = c.D / 8;
    const float none[8] = {__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""),
                           __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
    int from, to;
    if (j.beside && lost_tokens(c, j.b, from, to)) {
        E* z = static_cast<E*>(out.p) + (from * out.st + (int64_t)j.h * out.sh);
        for (int64_t i = threadIdx.x; i < (int64_t)(to - from) * chunks; i += kThreads)
            store8(z + i / chunks * out.st + 8 * (i % chunks), none);
    }
    if (!any) return;
    E* y = static_cast<E*>(out.p) + (j.t0 * out.st + (int64_t)j.h * out.sh);
    for (int64_t i = threadIdx.x; i < j.early * chunks; i += kThreads)
        store8(y + (i / chunks - j.early) * out.st + 8 * (i % chunks), none);
    if (!j.known) {
        for (int i = threadIdx.x; i < j.m * chunks; i += kThreads)
            store8(y + (int64_t)(i / chunks) * out.st + 8 * (i % chunks), none);
        return;
    }
    const float s = (j.values ? c.v_scale : c.k_scale)[j.row];
    const int8_t* pool = (j.values ? c.values : c.keys) + j.row * c.P * c.D;
    if (!j.values) {
#pragma unroll 4
        for (int i = threadIdx.x; i < j.m * chunks; i += kThreads) {
            const int tok = i / chunks, d = 8 * (i % chunks);
            union { uint2 w; int8_t b[8]; } u;
            u.w = *reinterpret_cast<const uint2*>(pool + (int64_t)(j.held + tok) * c.D + d);
            float e[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) e[q] = (float)u.b[q] * s;
            store8(y + (int64_t)tok * out.st + d, e);
        }
        return;
    }
    const int pitch = tile_pitch(c.P) / 4;
    const int p0 = j.held / 16, np = (j.held + j.m + 15) / 16 - p0;
#pragma unroll 4
    for (int i = threadIdx.x; i < np * c.D; i += kThreads) {
        const int d = i / np, t0 = 16 * (p0 + i % np);
        const uint4 w = *reinterpret_cast<const uint4*>(pool + (int64_t)d * c.P + t0);
        uint32_t* to = tile + d * pitch + t0 / 4;
        to[0] = w.x;
        to[1] = w.y;
        to[2] = w.z;
        to[3] = w.w;
    }
    __syncthreads();
    const int g0 = j.held / 4, n = ((j.held + j.m + 3) / 4 - g0) * chunks;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int g = g0 + i / chunks, tok = 4 * g - j.held, d = 8 * (i % chunks);
        uint32_t word[8];
#pragma unroll
        for (int p = 0; p < 8; ++p) word[p] = tile[(d + p) * pitch + g];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (tok + q < 0 || tok + q >= j.m) continue;
            float e[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) e[p] = (float)(int8_t)(word[p] >> (8 * q)) * s;
            store8(y + (int64_t)(tok + q) * out.st + d, e);
        }
    }
}

}  // namespace

hipError_t launch_cache_append(const CacheArgs& c, const Heads& k, const Heads& v, hipStream_t s) {
    const int per_seq = placed_by_tokens(c) ? 0 : (int)pages_touched(c.max_new, c.P);
    return launch_in_pieces(cache_copy_blocks(c), [&](uint32_t first, unsigned n) {
        if (c.dt == Dt::BF16) k_cache_append<uint16_t><<<n, kThreads, tile_bytes(c), s>>>(c, k, v, per_seq, first);
        else k_cache_append<float><<<n, kThreads, tile_bytes(c), s>>>(c, k, v, per_seq, first);
    });
}

hipError_t launch_cache_read(const CacheArgs& c, const Heads& k, const Heads& v, hipStream_t s) {
    const int per_seq = placed_by_tokens(c) ? 0 : (int)pages_touched(c.max_new, c.P);
    return launch_in_pieces(cache_copy_blocks(c), [&](uint32_t first, unsigned n) {
        if (c.dt == Dt::BF16) k_cache_read<uint16_t><<<n, kThreads, tile_bytes(c), s>>>(c, k, v, per_seq, first);
        else k_cache_read<float><<<n, kThreads, tile_bytes(c), s>>>(c, k, v, per_seq, first);
    });
}

}  // namespace sffn
