// Root-mean-square norm with the residual's addition, its outputs in 8 bits, and the
// gradient.
//
//   h = round(x + r),  y = h rsqrt(mean h^2 + eps) w
//   8 bits: n = h w, s = max|n| / top, entries round(n / s), scale s rsqrt(mean h^2 + eps)
//   gradient: u = g w, xh = h rstd, g_x = rstd (u - xh mean(u xh)) + g_h, g_w = sum g xh
//
// Memory-bound: everything is read and written once, the row stays in registers
// between the reduction and its use. 4096 bf16 rows of 4096: int8 25.2 us (117 MB, 4.7 TB/s),
// gradient 28.8 + 4.0 for the weight's sum (134 MB, 4.7 TB/s); one row 2.6 us.
#include <type_traits>

#include "attn_common.hpp"
#include "norm_launch.hpp"

namespace sffn {

namespace {

// 16 bytes of a row, aligned to whole elements only (rows of odd width or stride; the
// memory system takes dwordx4 accesses at any such address).
template <typename E>
struct Piece {
    static constexpr int N = 16 / sizeof(E);
    uint4 w;
    // the first n of the elements at p, zeros behind them
    __device__ __forceinline__ void load(const E* p, int n) {
        w = make_uint4(0, 0, 0, 0);
        if (n >= N) {
            __builtin_memcpy(&w, p, 16);
        } else if (n > 0) {
            E e[N] = {};
#pragma unroll
            for (int i = 0; i < N - 1; ++i)
                if (i < n) e[i] = p[i];
            __builtin_memcpy(&w, e, 16);
        }
    }
    __device__ __forceinline__ void get(float* v) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(E) == 2) {
                v[2 * i] = bf16_lo(u[i]);
                v[2 * i + 1] = bf16_hi(u[i]);
            } else {
                v[i] = __uint_as_float(u[i]);
            }
        }
    }
    __device__ __forceinline__ void set(const float* v) {
        if constexpr (sizeof(E) == 2)
            w = make_uint4(round2(v[0], v[1]), round2(v[2], v[3]), round2(v[4], v[5]), round2(v[6], v[7]));
        else
            w = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    __device__ __forceinline__ void store(E* p, int n) const {
        if (n >= N) {
            __builtin_memcpy(p, &w, 16);
        } else if (n > 0) {
            E e[N];
            __builtin_memcpy(e, &w, 16);
#pragma unroll
            for (int i = 0; i < N - 1; ++i)
                if (i < n) p[i] = e[i];
        }
    }
};

// N bytes to p, the first n of them.
template <int N>
__device__ __forceinline__ void store_bytes(uint8_t* p, const uint32_t (&w)[N / 4], int n) {
    if (n >= N) {
        __builtin_memcpy(p, w, N);
    } else {
#pragma unroll
        for (int i = 0; i < N - 1; ++i)
            if (i < n) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
    }
}

// Four entries of 8 bits of v / s.
template <NormOut OUT>
__device__ __forceinline__ uint32_t entries4(const float* v, float s) {
    constexpr float top = OUT == NormOut::Int8 ? 127.f : 448.f;
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        q[i] = s > 0.f ? v[i] / s : 0.f;        // IEEE division: the same entries wherever computed
        q[i] = fminf(fmaxf(q[i], -top), top);   // a scale below fp32's normal numbers is inexact
    }
    if constexpr (OUT == NormOut::Int8) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) w |= ((uint32_t)(int)rintf(q[i]) & 0xffu) << (8 * i);
        return w;
    } else {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    }
}

// The larger of two magnitudes, compared as integers, in which infinities and NaN come out
// on top (a floating-point maximum drops a NaN).
__device__ __forceinline__ float larger(float a, float b) {
    return __int_as_float(max(__float_as_int(a), __float_as_int(b)));
}

// The unit of a row's 8-bit entries, whose largest magnitude is `top`: NaN, and so the row's
// scale, where that is not finite.
template <NormOut OUT>
__device__ __forceinline__ float unit_of(float top) {
    return top < __builtin_huge_valf() ? top / (OUT == NormOut::Int8 ? 127.f : 448.f) : __builtin_nanf("");
}

// Sums (or largest magnitudes) over the NT threads of a row, the same in all of them: within
// waves, then across them in LDS in a fixed order. `at` is the row's place in LDS.
template <int NT, bool MAX>
__device__ __forceinline__ float2 row_reduce(float sum, float other, float2* at) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        sum += __shfl_xor(sum, o, 64);
        const float q = __shfl_xor(other, o, 64);
        other = MAX ? larger(other, q) : other + q;
    }
    if constexpr (NT > 64) {
        const int wave = threadIdx.x % NT / 64;
        if ((threadIdx.x & 63) == 0) at[wave] = make_float2(sum, other);
        __syncthreads();
        float2 v = at[0];
#pragma unroll
        for (int i = 1; i < NT / 64; ++i) {
            const float2 q = at[i];
            v.x += q.x;
            v.y = MAX ? larger(v.y, q.y) : v.y + q.y;
        }
        return v;
    }
    return make_float2(sum, other);
}

template <typename E>
__device__ __forceinline__ E* row_of(const Rows& v, int64_t t) { return static_cast<E*>(v.p) + t * v.stride; }

// ---------------------------------------------------------------------------
// Forward: NT threads a row, each with N pieces of 16 bytes.
// ---------------------------------------------------------------------------
constexpr int block_of(int NT) { return NT == 64 ? 256 : NT; }

template <typename E, int NT, int N, NormOut OUT>
__global__ __launch_bounds__(block_of(NT)) void k_norm(const NormArgs a) {
    constexpr int V = Piece<E>::N;
    __shared__ float2 lds[NT / 64];
    const int64_t t = a.first + (int64_t)blockIdx.x * (block_of(NT) / NT) + threadIdx.x / NT;
    if (t >= a.T) return;           // whole waves, and whole workgroups where they meet
    const int tid = threadIdx.x % NT;
    const E* px = row_of<const E>(a.x, t);
    const E* pr = a.r.p ? row_of<const E>(a.r, t) : nullptr;
    const E* pw = static_cast<const E*>(a.w);
    Piece<E> x[N], r[N], w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = (tid + i * NT) * V, n = a.d - at;
        x[i].load(px + at, n);
        if (pr) r[i].load(pr + at, n);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (pw) w[i].load(pw + (tid + i * NT) * V, a.d - (tid + i * NT) * V);
    float sum = 0.f, top = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = (tid + i * NT) * V, n = a.d - at;
        float h[V], q[V];
        x[i].get(h);
        if (pr) {
            r[i].get(q);
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] += q[j];
            x[i].set(h);
            x[i].get(h);
            if (a.h.p) x[i].store(row_of<E>(a.h, t) + at, n);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) sum += h[j] * h[j];
        if constexpr (OUT != NormOut::Same) {
            if (pw) {
                w[i].get(q);
#pragma unroll
                for (int j = 0; j < V; ++j) h[j] *= q[j];
            }
#pragma unroll
            for (int j = 0; j < V; ++j) top = larger(top, fabsf(h[j]));
        }
    }
    const float2 s = row_reduce<NT, true>(sum, top, lds);
    const float rstd = rsqrtf(s.x / a.d + a.eps);
    const float unit = unit_of<OUT>(s.y);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int at = (tid + i * NT) * V, n = a.d - at;
        float h[V], q[V];
        x[i].get(h);
        if (pw) {
            w[i].get(q);
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] *= q[j];
        }
        if constexpr (OUT == NormOut::Same) {
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] *= rstd;
            x[i].set(h);
            x[i].store(row_of<E>(a.y, t) + at, n);
        } else if (n > 0) {
            uint32_t e[V / 4];
#pragma unroll
            for (int j = 0; j < V; j += 4) e[j / 4] = entries4<OUT>(h + j, unit);
            store_bytes<V>(row_of<uint8_t>(a.y, t) + at, e, n);
        }
    }
    if (OUT != NormOut::Same && tid == 0) a.scale[t] = unit * rstd;
}

// Rows that no workgroup holds in its registers: read twice, a workgroup of 1024 a row.
template <typename E, NormOut OUT>
__global__ __launch_bounds__(1024) void k_norm_long(const NormArgs a) {
    constexpr int NT = 1024, V = Piece<E>::N;
    __shared__ float2 lds[NT / 64];
    const int64_t t = a.first + blockIdx.x;
    const E* px = row_of<const E>(a.x, t);
    const E* pr = a.r.p ? row_of<const E>(a.r, t) : nullptr;
    const E* pw = static_cast<const E*>(a.w);
    float sum = 0.f, top = 0.f;
    // the sum's piece at `at`, and times the weight
    auto value = [&](int at, float* h, float* nw) {
        const int n = a.d - at;
        Piece<E> x, q;
        x.load(px + at, n);
        x.get(h);
        if (pr) {
            float o[V];
            q.load(pr + at, n);
            q.get(o);
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] += o[j];
            x.set(h);
            x.get(h);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) nw[j] = h[j];
        if (pw) {
            float o[V];
            q.load(pw + at, n);
            q.get(o);
#pragma unroll
            for (int j = 0; j < V; ++j) nw[j] *= o[j];
        }
        return x;
    };
    for (int at = threadIdx.x * V; at < a.d; at += NT * V) {
        float h[V], nw[V];
        value(at, h, nw);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            sum += h[j] * h[j];
            top = larger(top, fabsf(nw[j]));
        }
    }
    const float2 s = row_reduce<NT, true>(sum, top, lds);
    const float rstd = rsqrtf(s.x / a.d + a.eps);
    const float unit = unit_of<OUT>(s.y);
    for (int at = threadIdx.x * V; at < a.d; at += NT * V) {
        const int n = a.d - at;
        float h[V], nw[V];
        Piece<E> x = value(at, h, nw);      // outputs that are inputs are written behind this thread's last read
        if (a.h.p) x.store(row_of<E>(a.h, t) + at, n);
        if constexpr (OUT == NormOut::Same) {
#pragma unroll
            for (int j = 0; j < V; ++j) nw[j] *= rstd;
            x.set(nw);
            x.store(row_of<E>(a.y, t) + at, n);
        } else {
            uint32_t e[V / 4];
#pragma unroll
            for (int j = 0; j < V; j += 4) e[j / 4] = entries4<OUT>(nw + j, unit);
            store_bytes<V>(row_of<uint8_t>(a.y, t) + at, e, n);
        }
    }
    if (OUT != NormOut::Same && threadIdx.x == 0) a.scale[t] = unit * rstd;
}

// ---------------------------------------------------------------------------
// Gradient: workgroups of B threads take B / NT rows at a time, the next ones' loads in
// flight (rows of up to 16 KB); the weight's gradient stays in registers over all of a
// workgroup's rows and leaves as one row of `partial`, added by k_norm_sum in a fixed order.
// ---------------------------------------------------------------------------
template <typename E, int NT, int N, int B>
__global__ __launch_bounds__(B) void k_norm_backward(const NormArgs a) {
    constexpr int V = Piece<E>::N, RB = B / NT;
    __shared__ float2 lds[2][B / 64];
    __shared__ float sums[RB > 1 ? NT * N * V : 1];
    const int tid = threadIdx.x % NT, group = threadIdx.x / NT;
    const E* pw = static_cast<const E*>(a.w);
    float gw[N][V];
    Piece<E> w[N], x[N], g[N], gh[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (pw) w[i].load(pw + (tid + i * NT) * V, a.d - (tid + i * NT) * V);
#pragma unroll
        for (int j = 0; j < V; ++j) gw[i][j] = 0.f;
    }
    auto load = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (tid + i * NT) * V, n = t < a.T ? a.d - at : 0;
            x[i].load(row_of<const E>(a.x, t) + at, n);
            g[i].load(row_of<const E>(a.g_y, t) + at, n);
            if (a.g_h.p) gh[i].load(row_of<const E>(a.g_h, t) + at, n);
        }
    };
    int64_t t0 = (int64_t)blockIdx.x * RB;
    constexpr bool ahead = N == 1;      // wider rows have no registers for the next one
    if (ahead) load(t0 + group);
    int turn = 0;
    for (; t0 < a.T; t0 += (int64_t)gridDim.x * RB, turn ^= 1) {
        const int64_t t = t0 + group;
        Piece<E> cx[N], cg[N], ch[N];
        float sum = 0.f, dot = 0.f;
        if (!ahead) load(t);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            cx[i] = x[i];
            cg[i] = g[i];
            ch[i] = gh[i];
        }
        if (ahead) load(t + (int64_t)gridDim.x * RB);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float h[V], u[V], q[V];
            cx[i].get(h);
            cg[i].get(u);
            if (pw) {
                w[i].get(q);
#pragma unroll
                for (int j = 0; j < V; ++j) u[j] *= q[j];
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                sum += h[j] * h[j];
                dot += u[j] * h[j];
            }
        }
        const float2 s = row_reduce<NT, false>(sum, dot, &lds[turn][group * (NT / 64)]);
        const float rstd = rsqrtf(s.x / a.d + a.eps);
        const float m = s.y * rstd / a.d;       // mean(u xh)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = (tid + i * NT) * V, n = t < a.T ? a.d - at : 0;
            float h[V], u[V], q[V];
            cx[i].get(h);
            cg[i].get(u);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                h[j] *= rstd;
                gw[i][j] += u[j] * h[j];
            }
            if (pw) {
                w[i].get(q);
#pragma unroll
                for (int j = 0; j < V; ++j) u[j] *= q[j];
            }
#pragma unroll
            for (int j = 0; j < V; ++j) u[j] = rstd * (u[j] - h[j] * m);
            if (a.g_h.p) {
                ch[i].get(q);
#pragma unroll
                for (int j = 0; j < V; ++j) u[j] += q[j];
            }
            cx[i].set(u);
            cx[i].store(row_of<E>(a.g_x, t) + at, n);
        }
    }
    if (!a.partial) return;
    float* out = a.partial + (int64_t)blockIdx.x * a.d;
    if constexpr (RB > 1) {
        for (int k = 0; k < RB; ++k) {
            if (group == k)
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        // by element and piece, so that the threads' words are consecutive
                        float& to = sums[(i * V + j) * NT + tid];
                        to = k == 0 ? gw[i][j] : to + gw[i][j];
                    }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < NT * N * V; c += B) {
            const int p = c / V, j = c % V, col = p * V + j;
            if (col < a.d) out[col] = sums[(p / NT * V + j) * NT + p % NT];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int col = (tid + i * NT) * V + j;
                if (col < a.d) out[col] = gw[i][j];
            }
    }
}

// Rows that no workgroup holds in its registers: read twice; the weight's gradient is
// kept in the workgroup's row of `partial`.
template <typename E>
__global__ __launch_bounds__(1024) void k_norm_backward_long(const NormArgs a) {
    constexpr int NT = 1024;
    __shared__ float2 lds[2][NT / 64];
    const E* pw = static_cast<const E*>(a.w);
    float* gw = a.partial ? a.partial + (int64_t)blockIdx.x * a.d : nullptr;
    auto get = [](const E* p) {
        if constexpr (sizeof(E) == 2) return bf16_to_f32(*p);
        else return *p;
    };
    int turn = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
        const E *px = row_of<const E>(a.x, t), *pg = row_of<const E>(a.g_y, t);
        float sum = 0.f, dot = 0.f;
        for (int i = threadIdx.x; i < a.d; i += NT) {
            const float h = get(px + i), u = get(pg + i) * (pw ? get(pw + i) : 1.f);
            sum += h * h;
            dot += u * h;
        }
        const float2 s = row_reduce<NT, false>(sum, dot, lds[turn]);
        const float rstd = rsqrtf(s.x / a.d + a.eps), m = s.y * rstd / a.d;
        for (int i = threadIdx.x; i < a.d; i += NT) {
            const float xh = get(px + i) * rstd, g = get(pg + i);
            if (gw) gw[i] = (t == blockIdx.x ? 0.f : gw[i]) + g * xh;
            float v = rstd * (g * (pw ? get(pw + i) : 1.f) - xh * m);
            if (a.g_h.p) v += get(row_of<const E>(a.g_h, t) + i);
            Elem<E>::store1(row_of<E>(a.g_x, t) + i, v);
        }
    }
}

// Sums of the columns of `partial` in a fixed order: 32 threads a column, each with
// every 32nd row.
constexpr int kSumCols = 32, kSumRows = 32;
__global__ __launch_bounds__(kSumCols* kSumRows) void k_norm_sum(const float* partial, int rows, int d, float* out) {
    __shared__ float lds[kSumRows][kSumCols];
    const int c = threadIdx.x % kSumCols, k = threadIdx.x / kSumCols;
    const int col = blockIdx.x * kSumCols + c;
    float v = 0.f;
    constexpr int IN = 8;           // loads in flight
    if (col < d)
        for (int r = k; r < rows; r += IN * kSumRows) {
            float x[IN];
#pragma unroll
            for (int i = 0; i < IN; ++i)
                x[i] = r + i * kSumRows < rows ? partial[(int64_t)(r + i * kSumRows) * d + col] : 0.f;
#pragma unroll
            for (int i = 0; i < IN; ++i) v += x[i];
        }
    lds[k][c] = v;
    __syncthreads();
    if (k != 0 || col >= d) return;
#pragma unroll
    for (int i = 1; i < kSumRows; ++i) v += lds[i][c];
    out[col] = v;
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
int pieces_of(const NormArgs& a) {
    const int per = a.dt == Dt::BF16 ? 8 : 4;
    return (a.d + per - 1) / per;
}

constexpr int64_t kMostNormBlocks = (int64_t)1 << 21;       // of up to 1024 threads: below 2^32 in a grid

template <typename F>
hipError_t in_pieces(const NormArgs& a, int rows_each, F launch) {
    const int64_t blocks = (a.T + rows_each - 1) / rows_each;
    for (int64_t first = 0; first < blocks; first += kMostNormBlocks) {
        NormArgs piece = a;
        piece.first = first * rows_each;
        launch(piece, (unsigned)(blocks - first < kMostNormBlocks ? blocks - first : kMostNormBlocks));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename E, NormOut OUT, int NT, int N>
hipError_t forward(const NormArgs& a, hipStream_t s) {
    return in_pieces(a, block_of(NT) / NT, [&](const NormArgs& p, unsigned n) {
        k_norm<E, NT, N, OUT><<<dim3(n), block_of(NT), 0, s>>>(p);
    });
}

// One piece a thread as far as a workgroup goes: bf16 rows of 8192 by 1024 threads take 3.2
// us for one and 22.9 for 2048 of them (134 MB, in part from the last-level cache), by 512
// of two pieces 3.6 and 22.8, by 256 of four 4.5 and 23.5; rows of 16384 by 1024 of two
// pieces 4.1, by 512 of four 4.9. (Rows of 32768 held 5.9, read twice 8.5.)
template <typename E, NormOut OUT>
hipError_t forward_by_width(const NormArgs& a, hipStream_t s) {
    const int p = pieces_of(a);
    if (p <= 64) return forward<E, OUT, 64, 1>(a, s);
    if (p <= 128) return forward<E, OUT, 128, 1>(a, s);
    if (p <= 256) return forward<E, OUT, 256, 1>(a, s);
    if (p <= 512) return forward<E, OUT, 512, 1>(a, s);
    if (p <= 1024) return forward<E, OUT, 1024, 1>(a, s);
    if (p <= 2048) return forward<E, OUT, 1024, 2>(a, s);
    if (p <= 4096) return forward<E, OUT, 1024, 4>(a, s);
    return in_pieces(a, 1, [&](const NormArgs& q, unsigned n) { k_norm_long<E, OUT><<<dim3(n), 1024, 0, s>>>(q); });
}

template <typename E>
hipError_t forward_by_output(const NormArgs& a, hipStream_t s) {
    switch (a.out) {
        case NormOut::Int8: return forward_by_width<E, NormOut::Int8>(a, s);
        case NormOut::E4m3: return forward_by_width<E, NormOut::E4m3>(a, s);
        default: return forward_by_width<E, NormOut::Same>(a, s);
    }
}

// Threads of a row of the gradient, one piece each up to 1024 of them, in workgroups of 1024,
// one a compute unit: 32768 bf16 rows of 512 take 26.8 us with the sum behind it, in
// workgroups of 512 threads 31.6, of 256 49.2; 4096 rows of 4096 29.7, in workgroups of 512
// 38.3, with two pieces a thread 45.6; 2048 rows of 8192 34.0, with two pieces 41.8. (One row
// of 512 took 7.3 us so with a sum behind it, in a workgroup of 256 5.5.) Rows of 16384 by 512 threads of four
// pieces 42.1, by 1024 of two 45.7, read twice 103.
int backward_threads(int p) { return p <= 64 ? 64 : p <= 128 ? 128 : p <= 256 ? 256 : p <= 512 ? 512 : 1024; }

int64_t backward_rows_each(const NormArgs& a) { return 1024 / backward_threads(pieces_of(a)); }

// The rows of one or two turns go to one workgroup, whose sums are the weight's gradient: no
// second launch (rows of 4096: one turn 5.0 us, by two launches 7.0; two 6.7 and 7.1, three
// 8.3 and 7.2).
constexpr int64_t kTurnsAlone = 2;
int64_t backward_grid(const NormArgs& a) {
    const int64_t each = backward_rows_each(a), blocks = (a.T + each - 1) / each, most = compute_units();
    return blocks <= kTurnsAlone ? 1 : blocks < most ? blocks : most;
}

template <typename E>
hipError_t backward(const NormArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)backward_grid(a));
    const int p = pieces_of(a);
    if (p <= 64) k_norm_backward<E, 64, 1, 1024><<<grid, 1024, 0, s>>>(a);
    else if (p <= 128) k_norm_backward<E, 128, 1, 1024><<<grid, 1024, 0, s>>>(a);
    else if (p <= 256) k_norm_backward<E, 256, 1, 1024><<<grid, 1024, 0, s>>>(a);
    else if (p <= 512) k_norm_backward<E, 512, 1, 1024><<<grid, 1024, 0, s>>>(a);
    else if (p <= 1024) k_norm_backward<E, 1024, 1, 1024><<<grid, 1024, 0, s>>>(a);
    else if (p <= 2048) k_norm_backward<E, 512, 4, 512><<<grid, 512, 0, s>>>(a);
    else if (sizeof(E) == 4 && p <= 4096) k_norm_backward<float, 1024, 4, 1024><<<grid, 1024, 0, s>>>(a);
    else k_norm_backward_long<E><<<grid, 1024, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t norm_partial_rows(const NormArgs& a) { return backward_grid(a); }

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
    return a.dt == Dt::BF16 ? forward_by_output<uint16_t>(a, s) : forward_by_output<float>(a, s);
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t s) {
    const int64_t rows = backward_grid(a);
    NormArgs b = a;
    if (rows == 1 && a.g_w) b.partial = a.g_w;
    const hipError_t e = a.dt == Dt::BF16 ? backward<uint16_t>(b, s) : backward<float>(b, s);
    if (e != hipSuccess || !a.g_w || rows == 1) return e;
    k_norm_sum<<<dim3((unsigned)((a.d + kSumCols - 1) / kSumCols)), kSumCols * kSumRows, 0, s>>>(
        a.partial, (int)rows, a.d, a.g_w);
    return hipGetLastError();
}

}  // namespace sffn
