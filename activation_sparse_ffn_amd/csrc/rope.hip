// Norms of q and k for each head and the rotation of their pairs by position,
// in one pass over the data, and its gradient.
//
//   n = x r w, r = rsqrt(mean x^2 + eps)     y_a = n_a c - n_b s, y_b = n_b c + n_a s
//
// Gradient, with g = dL/dy and x^ = x r: the rotation is orthogonal, so gn is g
// turned back (s -> -s); dL/dw = sum over tokens and heads of gn x^; with u = w
// gn, dL/dx = r (u - x^ mean(u x^)).
//
// Memory-bound: 2 bytes moved and 8 to 14 operations per element and byte, so
// the whole head stays in registers between its one read and its one write. A
// head is held by a group of LH lanes, eight elements (16 bytes of bf16) each,
// so that the norm's sum is log2 LH exchanges and a pair's other half is at
// most one exchange away. A group takes several heads of one token in turn and
// keeps that token's cos and sin (64 bytes a lane, four times a head's own
// bytes) in registers.
#include <type_traits>

#include "attn_common.hpp"
#include "attn_launch.hpp"

namespace sffn {

namespace {

constexpr int kThreads = 256;

template <typename E> __device__ __forceinline__ float to_f32(E v);
template <> __device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return bf16_to_f32(v); }
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }

template <int LH>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = LH / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o, LH);
    return v;
}

// cos and sin of a lane's eight elements, set up once per token. Half layout:
// element i of the first half turns with element i + R/2 (own = c, other = -s),
// one of the second half with i - R/2 (other = +s). Interleaved: pairs lie
// inside the lane, four angles.
struct Angles {
    float c[8], s[8];
};

// dir = +1: forward; -1: the rotation turned back
__device__ __forceinline__ Angles load_angles(const RopeArgs& a, int32_t pos, int c8, float dir) {
    Angles t;
    if (8 * c8 >= a.R) return t;       // not rotated, never used
    const float* row = a.table + (size_t)pos * a.R;
    const int half = a.R / 2;
    if (a.interleaved) {
        const float4 c = *reinterpret_cast<const float4*>(row + 4 * c8);
        const float4 s = *reinterpret_cast<const float4*>(row + half + 4 * c8);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            t.c[i] = cc[i / 2];
            t.s[i] = (i & 1) ? dir * ss[i / 2] : -dir * ss[i / 2];
        }
    } else {
        const bool second = 8 * c8 >= half;
        const float* p = row + 8 * c8 - (second ? half : 0);
        const float sign = second ? dir : -dir;
        Elem<float>::load8(p, t.c);
        Elem<float>::load8(p + half, t.s);
#pragma unroll
        for (int i = 0; i < 8; ++i) t.s[i] *= sign;
    }
    return t;
}

// y = n c + (n of the pair's other element) s, for rotated lanes
template <int LH>
__device__ __forceinline__ void turn(const RopeArgs& a, const Angles& t, int c8, float* n) {
    if (a.R == 0) return;
    const bool rotated = 8 * c8 < a.R;
    if (a.interleaved) {
        if (!rotated) return;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float x = n[i], y = n[i + 1];
            n[i] = x * t.c[i] + y * t.s[i];
            n[i + 1] = y * t.c[i + 1] + x * t.s[i + 1];
        }
    } else {
        const int hc = a.R / 16;
        const int other = rotated ? (c8 < hc ? c8 + hc : c8 - hc) : c8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = __shfl(n[i], other, LH);
            if (rotated) n[i] = n[i] * t.c[i] + o * t.s[i];
        }
    }
}

__device__ __forceinline__ size_t at(const Heads& v, int64_t t, int h) {
    return (size_t)(t * v.st + (int64_t)h * v.sh);
}

// Row of head h (q's heads, then k's) of token t in the views of q and k.
template <typename E>
__device__ __forceinline__ E* row_of(const RopeArgs& a, const Heads& q, const Heads& k, int64_t t, int h) {
    const bool is_q = h < a.n_q;
    return static_cast<E*>(is_q ? q.p : k.p) + (is_q ? at(q, t, h) : at(k, t, h - a.n_q));
}

// ---------------------------------------------------------------------------
// forward, 16-byte accesses: D and the strides multiples of eight, R of 16
// (half layout) or 8 (interleaved), 16-byte aligned data. Group g of the grid
// takes heads s, s + per, ... of token t, where g = t per + s, the next head's
// load in flight. (Four heads' loads at once cost more in waves than they gave:
// 24.9 against 22.4 us for a 4096-token chunk of 40 heads of 128, which takes
// 19.4 us, 4.4 TB/s, with 31-bit indexes.) One token takes 3.3 us, the launch.
// ---------------------------------------------------------------------------
template <typename E, int LH>
__global__ __launch_bounds__(kThreads) void k_rope(const RopeArgs a, int per) {
    const int c8 = threadIdx.x & (LH - 1);
    const int64_t g = (int64_t)blockIdx.x * (kThreads / LH) + threadIdx.x / LH;
    const int64_t t = g / per;
    if (t >= a.T) return;
    const int s = (int)(g - t * per);
    const int heads = a.n_q + a.n_k;
    const bool have = 8 * c8 < a.D;
    bool ok = true;
    Angles ang;
    if (a.R > 0) {
        const int32_t pos = a.pos[t];
        ok = pos >= 0 && pos < a.max_pos;
        ang = load_angles(a, ok ? pos : 0, c8, 1.f);
    }
    Raw<E> next;
    if (have) next.load(row_of<E>(a, a.q, a.k, t, s) + 8 * c8);
    for (int h = s; h < heads; h += per) {
        const bool is_q = h < a.n_q;
        const Raw<E> raw = next;
        if (have && h + per < heads) next.load(row_of<E>(a, a.q, a.k, t, h + per) + 8 * c8);
        float n[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = 0.f;
        if (have) raw.decode(n);
        if (a.norm) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.f;
            const E* wp = static_cast<const E*>(is_q ? a.q_w : a.k_w);
            if (wp && have) Elem<E>::load8(wp + 8 * c8, w);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += n[i] * n[i];
            const float r = rsqrtf(group_sum<LH>(sum) / (float)a.D + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] *= r * w[i];
        }
        turn<LH>(a, ang, c8, n);
        if (!ok)
#pragma unroll
            for (int i = 0; i < 8; ++i) n[i] = __builtin_nanf("");
        if (have) store8(row_of<E>(a, a.q_out, a.k_out, t, h) + 8 * c8, n);
    }
}

// ---------------------------------------------------------------------------
// backward, same conditions. A workgroup walks groups of the grid with a
// stride of the whole grid and keeps its share of the weights' gradients in
// registers (a lane's eight channels of q and of k); the groups of a workgroup
// meet in LDS and leave one row of `partial` [blocks, 2, D], which k_rope_sum
// adds in a fixed order. (A 4096-token chunk of 40 heads of 128: 28.7 us, 126 MB
// at 4.4 TB/s.)
// ---------------------------------------------------------------------------
template <typename E, int LH>
__global__ __launch_bounds__(kThreads) void k_rope_backward(const RopeArgs a, int per) {
    constexpr int GB = kThreads / LH;
    const int c8 = threadIdx.x & (LH - 1), gl = threadIdx.x / LH;
    const int heads = a.n_q + a.n_k;
    const bool have = 8 * c8 < a.D;
    const int64_t groups = a.T * per;
    float wq[8], wk[8], sq[8], sk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        wq[i] = wk[i] = 1.f;
        sq[i] = sk[i] = 0.f;
    }
    if (a.norm && have) {
        if (a.q_w) Elem<E>::load8(static_cast<const E*>(a.q_w) + 8 * c8, wq);
        if (a.k_w) Elem<E>::load8(static_cast<const E*>(a.k_w) + 8 * c8, wk);
    }
    for (int64_t g = (int64_t)blockIdx.x * GB + gl; g < groups; g += (int64_t)gridDim.x * GB) {
        const int64_t t = g / per;
        bool ok = true;
        Angles ang;
        if (a.R > 0) {
            const int32_t pos = a.pos[t];
            ok = pos >= 0 && pos < a.max_pos;
            ang = load_angles(a, ok ? pos : 0, c8, -1.f);
        }
        Raw<E> next_g, next_x;
        auto load = [&](int h) {
            if (!have) return;
            next_g.load(row_of<E>(a, a.g_q, a.g_k, t, h) + 8 * c8);
            if (a.norm) next_x.load(row_of<E>(a, a.q, a.k, t, h) + 8 * c8);
        };
        load((int)(g - t * per));
        for (int h = (int)(g - t * per); h < heads; h += per) {
            const bool is_q = h < a.n_q;
            const Raw<E> raw_g = next_g, raw_x = next_x;
            if (h + per < heads) load(h + per);
            float gn[8], x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) gn[i] = x[i] = 0.f;
            if (have) {
                raw_g.decode(gn);
                if (a.norm) raw_x.decode(x);
            }
            turn<LH>(a, ang, c8, gn);
            if (!ok)
#pragma unroll
                for (int i = 0; i < 8; ++i) gn[i] = __builtin_nanf("");
            if (a.norm) {
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += x[i] * x[i];
                const float r = rsqrtf(group_sum<LH>(sum) / (float)a.D + a.eps);
                float dot = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] *= r;
                    const float gw = gn[i] * x[i];
                    if (is_q) sq[i] += gw; else sk[i] += gw;
                    gn[i] *= is_q ? wq[i] : wk[i];
                    dot += have ? gn[i] * x[i] : 0.f;
                }
                const float m = group_sum<LH>(dot) / (float)a.D;
#pragma unroll
                for (int i = 0; i < 8; ++i) gn[i] = r * (gn[i] - x[i] * m);
            }
            if (have) store8(row_of<E>(a, a.q_out, a.k_out, t, h) + 8 * c8, gn);
        }
    }
    if (!a.norm || !a.partial) return;
    __shared__ float lds[kThreads * 8];
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
#pragma unroll
        for (int i = 0; i < 8; ++i) lds[gl * (8 * LH) + 8 * c8 + i] = part ? sk[i] : sq[i];
        __syncthreads();
        for (int d = threadIdx.x; d < a.D; d += kThreads) {
            float sum = 0.f;
            for (int j = 0; j < GB; ++j) sum += lds[j * (8 * LH) + d];
            a.partial[((size_t)blockIdx.x * 2 + part) * a.D + d] = sum;
        }
        __syncthreads();
    }
}

// Columns of partial [n, 2 D] summed: 64 threads a column, each every 64th row
// with eight loads in flight, joined in order. (With 16 threads a column and one
// load at a time the 1024 rows of a 4096-token chunk took 20 us, now 3.9.)
constexpr int kSumRows = 64;

__global__ __launch_bounds__(16 * kSumRows) void k_rope_sum(const float* __restrict__ partial, int n, int D,
                                                            float* g_qw, float* g_kw) {
    __shared__ float lds[kSumRows][17];
    const int c = threadIdx.x & 15, r = threadIdx.x >> 4;
    const int col = blockIdx.x * 16 + c;
    float sum = 0.f;
    if (col < 2 * D && r < n)
        sum = sum_splits_in_order(partial + (size_t)r * 2 * D + col, (n - r + kSumRows - 1) / kSumRows,
                                  (int64_t)kSumRows * 2 * D);
    lds[r][c] = sum;
    __syncthreads();
    if (r < 8) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kSumRows / 8; ++i) sum += lds[r + 8 * i][c];
    }
    __syncthreads();
    if (r < 8) lds[r][c] = sum;
    __syncthreads();
    if (r == 0 && col < 2 * D) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += lds[i][c];
        float* to = col < D ? g_qw : g_kw;
        if (to) to[col < D ? col : col - D] = sum;
    }
}

// ---------------------------------------------------------------------------
// any head_dim <= 512, any even R, any strides: a wave per head, lane l holds
// elements l, l + 64, .... A pair's other element is read from memory as well,
// before anything is written, so an output may be its own input.
//
// It takes what the 16-byte kernels do not (see wide): heads of a size that eight
// does not divide, rotated parts that do not fill eights of both halves, rows that
// are not 16-byte aligned. Each element is read twice, 2 or 4 bytes at a time, and
// the table's row again for every head: 4096 tokens of 40 heads of 80, 40 of them
// rotated in halves, take 112 us, their gradient 158 + 4.6 (with 32 rotated, by the
// 16-byte kernels, 18.7 and 26 + 4.0).
//
// The gradient's difference u - x^ mean(u x^) cancels where u is nearly along x^,
// most of all in heads of a few elements (with one it leaves eps r^2 of its terms);
// those of fewer than eight come here. So this kernel takes r, x^, the mean and the
// difference in 64 bits.
// ---------------------------------------------------------------------------
constexpr int kPer = 8;     // 512 / 64

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}

template <typename E, bool BWD>
__global__ __launch_bounds__(kThreads) void k_rope_any(const RopeArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int heads = a.n_q + a.n_k;
    const int64_t units = a.T * heads;
    float sq[kPer], sk[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) sq[i] = sk[i] = 0.f;
    for (int64_t u = (int64_t)blockIdx.x * 4 + wave; u < units; u += (int64_t)gridDim.x * 4) {
        const int64_t t = u / heads;
        const int h = (int)(u - t * heads);
        const bool is_q = h < a.n_q;
        const int hh = is_q ? h : h - a.n_q;
        const Heads& in = is_q ? a.q : a.k;
        const Heads& turned = BWD ? (is_q ? a.g_q : a.g_k) : in;
        const Heads& out = is_q ? a.q_out : a.k_out;
        const E* xp = static_cast<const E*>(in.p) + (BWD && !a.norm ? 0 : at(in, t, hh));
        const E* tp = static_cast<const E*>(turned.p) + at(turned, t, hh);
        const E* wp = a.norm ? static_cast<const E*>(is_q ? a.q_w : a.k_w) : nullptr;
        int32_t pos = 0;
        bool ok = true;
        if (a.R > 0) {
            pos = a.pos[t];
            ok = pos >= 0 && pos < a.max_pos;
            if (!ok) pos = 0;
        }
        const float* row = a.table + (size_t)pos * a.R;
        // own[i], other[i]: element e and its pair's other one of what is turned
        float x[kPer], own[kPer], other[kPer], w[kPer], wo[kPer];
        typedef std::conditional_t<BWD, double, float> Acc;
        Acc sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 64 * i;
            x[i] = own[i] = other[i] = 0.f;
            w[i] = wo[i] = 1.f;
            if (e >= a.D) continue;
            int o = e;
            if (e < a.R) o = a.interleaved ? e ^ 1 : (e < a.R / 2 ? e + a.R / 2 : e - a.R / 2);
            own[i] = to_f32<E>(tp[e]);
            other[i] = to_f32<E>(tp[o]);
            if (a.norm) x[i] = BWD ? to_f32<E>(xp[e]) : own[i];
            if (wp) { w[i] = to_f32<E>(wp[e]); wo[i] = to_f32<E>(wp[o]); }
            sum += (Acc)x[i] * x[i];
        }
        Acc r = 1;
        if (a.norm) {
            if constexpr (BWD) r = 1.0 / sqrt(wave_sum64(sum) / a.D + (double)a.eps);
            else r = rsqrtf(wave_sum(sum) / (float)a.D + a.eps);
        }
        Acc dot = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 64 * i;
            if (e >= a.D) continue;
            float v = own[i], vo = other[i];
            if (!BWD) { v *= r * w[i]; vo *= r * wo[i]; }
            if (e < a.R) {
                const bool first = a.interleaved ? (e & 1) == 0 : e < a.R / 2;
                const int idx = a.interleaved ? e / 2 : (first ? e : e - a.R / 2);
                const float c = row[idx], s = row[a.R / 2 + idx];
                v = v * c + vo * (first != BWD ? -s : s);
            }
            if (!ok) v = __builtin_nanf("");
            if (BWD && a.norm) {
                const Acc xh = x[i] * r;
                const float gw = (float)(v * xh);
                if (is_q) sq[i] += gw; else sk[i] += gw;
                v *= w[i];
                dot += v * xh;
            }
            own[i] = v;
        }
        Acc m = 0;
        if constexpr (BWD)
            if (a.norm) m = wave_sum64(dot) / a.D;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int e = lane + 64 * i;
            if (e >= a.D) continue;
            const float v = BWD && a.norm ? (float)(r * (own[i] - x[i] * r * m)) : own[i];
            Elem<E>::store1(static_cast<E*>(out.p) + at(out, t, hh) + e, v);
        }
    }
    if (!BWD || !a.norm || !a.partial) return;
    __shared__ float lds[4][64 * kPer];
#pragma unroll 1
    for (int part = 0; part < 2; ++part) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) lds[wave][lane + 64 * i] = part ? sk[i] : sq[i];
        __syncthreads();
        for (int d = threadIdx.x; d < a.D; d += kThreads)
            a.partial[((size_t)blockIdx.x * 2 + part) * a.D + d] = lds[0][d] + lds[1][d] + lds[2][d] + lds[3][d];
        __syncthreads();
    }
}

bool wide_view(const Heads& v) {
    return v.p == nullptr || ((reinterpret_cast<uintptr_t>(v.p) & 15) == 0 && v.st % 8 == 0 && v.sh % 8 == 0);
}

// whether the 16-byte kernels apply (see k_rope)
bool wide(const RopeArgs& a) {
    auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    return a.D % 8 == 0 && a.R % (a.interleaved ? 8 : 16) == 0 && wide_view(a.q) && wide_view(a.k) &&
           wide_view(a.g_q) && wide_view(a.g_k) && wide_view(a.q_out) &&
           wide_view(a.k_out) && al(a.table) && al(a.q_w) && al(a.k_w);
}

int lanes_per_head(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : 64; }

// Groups of lanes for each token: one per head for few tokens (latency), one
// for every four heads or so where the grid fills the chip anyway.
int groups_per_token(const RopeArgs& a) {
    const int heads = a.n_q + a.n_k;
    const int64_t lanes = a.T * heads * lanes_per_head(a.D);
    if (lanes < (int64_t)compute_units() * 2048) return heads;
    return (heads + 3) / 4;
}

constexpr int kBackwardBlocks = 1024;

int64_t backward_blocks(const RopeArgs& a) {
    const int64_t rows = a.T * (a.n_q + a.n_k);
    const int64_t per_block = wide(a) ? kThreads / lanes_per_head(a.D) : 4;
    const int64_t blocks = (rows + per_block - 1) / per_block;
    return blocks < kBackwardBlocks ? blocks : kBackwardBlocks;
}

// A forward of tokens t .. t + n - 1 alone.
template <typename E>
RopeArgs tokens_of(const RopeArgs& a, int64_t t, int64_t n) {
    RopeArgs b = a;
    b.T = n;
    if (b.pos) b.pos += t;
    for (Heads* v : {&b.q, &b.k, &b.q_out, &b.k_out})
        if (v->p) v->p = static_cast<E*>(v->p) + t * v->st;
    return b;
}

template <typename E>
hipError_t launch_wide(const RopeArgs& a, hipStream_t s) {
    const int per = groups_per_token(a), LH = lanes_per_head(a.D);
    const int64_t groups = a.T * per, gb = kThreads / LH;
    if ((groups + gb - 1) / gb > kMostBlocks) {
        // more than a grid holds: tokens in two halves
        const int64_t t = a.T / 2;
        const hipError_t e = launch_wide<E>(tokens_of<E>(a, 0, t), s);
        return e != hipSuccess ? e : launch_wide<E>(tokens_of<E>(a, t, a.T - t), s);
    }
    const dim3 grid((unsigned)((groups + gb - 1) / gb));
    if (LH == 8) k_rope<E, 8><<<grid, kThreads, 0, s>>>(a, per);
    else if (LH == 16) k_rope<E, 16><<<grid, kThreads, 0, s>>>(a, per);
    else if (LH == 32) k_rope<E, 32><<<grid, kThreads, 0, s>>>(a, per);
    else k_rope<E, 64><<<grid, kThreads, 0, s>>>(a, per);
    return hipGetLastError();
}

template <typename E>
hipError_t launch_wide_backward(const RopeArgs& a, hipStream_t s) {
    const int per = groups_per_token(a), LH = lanes_per_head(a.D);
    const dim3 grid((unsigned)backward_blocks(a));
    if (LH == 8) k_rope_backward<E, 8><<<grid, kThreads, 0, s>>>(a, per);
    else if (LH == 16) k_rope_backward<E, 16><<<grid, kThreads, 0, s>>>(a, per);
    else if (LH == 32) k_rope_backward<E, 32><<<grid, kThreads, 0, s>>>(a, per);
    else k_rope_backward<E, 64><<<grid, kThreads, 0, s>>>(a, per);
    return hipGetLastError();
}

template <bool BWD>
hipError_t launch_any(const RopeArgs& a, hipStream_t s) {
    int64_t blocks = BWD ? backward_blocks(a) : (a.T * (a.n_q + a.n_k) + 3) / 4;
    if (blocks > kMostBlocks) blocks = kMostBlocks;         // waves then take several heads
    if (a.dt == Dt::BF16) k_rope_any<uint16_t, BWD><<<dim3((unsigned)blocks), kThreads, 0, s>>>(a);
    else k_rope_any<float, BWD><<<dim3((unsigned)blocks), kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t rope_partial_floats(const RopeArgs& a) { return a.norm ? (size_t)kBackwardBlocks * 2 * a.D : 0; }

hipError_t launch_rope(const RopeArgs& a, hipStream_t s) {
    if (!wide(a)) return launch_any<false>(a, s);
    return a.dt == Dt::BF16 ? launch_wide<uint16_t>(a, s) : launch_wide<float>(a, s);
}

hipError_t launch_rope_backward(const RopeArgs& a, hipStream_t s) {
    hipError_t e;
    if (!wide(a)) e = launch_any<true>(a, s);
    else e = a.dt == Dt::BF16 ? launch_wide_backward<uint16_t>(a, s) : launch_wide_backward<float>(a, s);
    if (e != hipSuccess || !a.norm || !a.partial) return e;
    k_rope_sum<<<dim3((2 * a.D + 15) / 16), 16 * kSumRows, 0, s>>>(a.partial, (int)backward_blocks(a), a.D, a.g_qw, a.g_kw);
    return hipGetLastError();
}

}  // namespace sffn
