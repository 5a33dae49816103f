// Attention of new tokens over the paged 4-bit cache.
//
//   s_j = scale q . k_j,  o = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - max),
//   k_j = entries times 2^e of each 32 channels,  v_j = entries times a scale sv_j
//
// One pass over the keys with the running maximum m and sum l of the softmax, S^T = K Q^T
// and O^T = V^T P^T as over the 8-bit cache, so that weights stay in the lanes that
// computed them. Entries are operands of the matrix cores as they lie:
// v_mfma_scale_f32_*_f8f6f4 multiplies 4-bit rows by 6-bit columns (1 sign, 2 exponent, 3
// mantissa bits: 0.125 .. 7.5) with a power of two for each 32 elements of either, which is
// what the keys' exponents are.
//
// q (times scale log2 e, or its power of two alone: see whole_q) and the weights p sv are
// sums of such 6-bit pieces: the block's
// largest magnitude goes to (3.75, 7.5] units, and each piece takes what the pieces before
// left, at 1 / 16 of their unit. The first leaves a quarter of a unit at most (rounding
// among steps of 1 / 2), the second 2^-7 (a quarter is 4 of its units, below which steps
// are 1 / 4), the third 2^-12 (2 of its units, steps of 1 / 8), each more 2^-4 of that:
// three pieces are exact to 2^-13.9 of the block's largest, four to 2^-17.9, five to
// 2^-21.9. Where there are but two, the second's unit is 1 / 32 of the first's: what the
// few largest elements leave may pass its range (they are exact to 2^-6 units, 2^-7.9 of
// the largest), the many below a quarter of the largest are so to 2^-9 units, half of what
// 1 / 16 leaves. q's blocks are 32 channels of a row, the weights' the 32 keys of a row that
// a lane holds. q of bf16 has four pieces, of fp32 five; weights two in sequences of more
// than kPreciseRows rows, three in those of fewer, five for fp32. The sum l takes the
// weights before they are cut. (4096 tokens over 32768 keys, 1.90 ms on one card: with three
// pieces of the weights 2.21, error 1.7e-3 instead of 2.1e-3; with three of q 1.78, but they
// hold a bf16 entry whole only down to 2^-6 of the largest of 32.)
#include <type_traits>
#include <utility>

#include "attn_work.hpp"

namespace sffn {

namespace {

struct Attn4Args {
    AttnArgs a;
    Cache4 b;
};

// The kernel's arguments once more, read where this is called: what only a work's end needs
// would be kept in spilled scalars during its loop.
__device__ __forceinline__ AttnArgs late_args() {
    auto p = (const __attribute__((address_space(4))) char*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    AttnArgs a;
    __builtin_memcpy(&a, (const void*)(p + offsetof(Attn4Args, a)), sizeof a);
    return a;
}

typedef uint32_t u32x6 __attribute__((ext_vector_type(6)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x32 __attribute__((ext_vector_type(32)));

template <typename F, int... I>
__device__ __forceinline__ void each(F f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
// f(0) .. f(N - 1), constants
template <int N, typename F>
__device__ __forceinline__ void each(F f) {
    each(f, std::make_integer_sequence<int, N>{});
}

// ---- 6-bit pieces ---------------------------------------------------------------

// A piece's unit is 2^-ratio of the one's before.
constexpr int ratio_of(int NP) { return NP == 2 ? 5 : 4; }

// Exponent (plus 127) of the unit of a block whose largest magnitude has the bits `top`:
// that lies in (3.75, 7.5] units. 255, which is NaN to the matrix cores, where it is not
// finite. The last of NP pieces' units is still a normal number.
template <int NP>
__device__ __forceinline__ int unit_of(uint32_t top) {
    const int e = (int)((top + 0x0fffffu) >> 23) - 2;
    return top >= 0x7f800000u ? 255 : max(e, ratio_of(NP) * (NP - 1) + 1);
}
// The units of NP pieces, a byte each, in two words.
template <int NP>
__device__ __forceinline__ void units(int e, int (&u)[2]) {
    constexpr uint32_t r = ratio_of(NP), steps = r << 8 | 2 * r << 16 | 3 * r << 24;
    u[0] = e == 255 ? -1 : (int)((uint32_t)e * 0x01010101u - steps);
    u[1] = NP <= 4 ? 0 : e == 255 ? -1 : e - 4 * (int)r;
}

// 32 numbers as NP pieces, the first of unit 2^(e - 127): element 2 j is lo[j], 2 j + 1
// hi[j]. The conversions write their result while they still read their operands: the empty
// asm keeps those, the unit among them, in other registers. (With the result over an operand
// the pieces were wrong.)
template <int NP>
__device__ __forceinline__ void split(f32x16 lo, f32x16 hi, int e, u32x6* out) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const float unit = __uint_as_float((uint32_t)(e - ratio_of(NP) * p) << 23);
        u32x6 r = __builtin_amdgcn_cvt_scalef32_2xpk16_fp6_f32(lo, hi, unit);
        asm("" : "+v"(r) : "v"(lo), "v"(hi), "v"(unit));
        out[p] = r;
        if (p + 1 < NP) {
            f32x32 back = __builtin_amdgcn_cvt_scalef32_pk32_f32_fp6(r, unit);
            asm("" : "+v"(back) : "v"(r), "v"(unit));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                lo[i] -= back[2 * i];
                hi[i] -= back[2 * i + 1];
            }
        }
    }
}

// 32 consecutive channels of a row of q, as they lie.
template <typename E>
struct QBlock {
    Raw<E> x[4];
    bool valid;
    __device__ __forceinline__ void load(const E* p, bool row) {
        valid = row;
        if (row)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i].load(p + 8 * i);
    }
    // times `by`, as NP pieces: their units' exponent
    template <int NP>
    __device__ __forceinline__ int split_into(float by, u32x6* out) const {
        float v[32];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i].decode(v + 8 * i);
#pragma unroll
            for (int j = 8 * i; j < 8 * i + 8; ++j) {
                v[j] = valid ? v[j] * by : 0.f;
                top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
            }
        }
        const int e = unit_of<NP>(top);
        f32x16 lo, hi;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            lo[i] = v[2 * i];
            hi[i] = v[2 * i + 1];
        }
        split<NP>(lo, hi, e, out);
        return e;
    }
};

// What of scale log2 e is multiplied into q before it is cut, and what is left for the scores.
// WHOLE: the power of two alone goes into q. The four pieces then hold a bf16 q's own entries,
// exactly those down to 2^-10 of the largest of 32, where its products with the scale are off by
// up to 2^-17.9 of it (the logarithm of a sum over one key by 4e-6 of itself, instead of 1e-7).
struct Scaling {
    float q, s;
};
// The rest costs a multiplication a score, which the few-row kernels have time for. The row
// tiles of heads of 128 need the registers that the reference as the products' third operand
// takes: 4096 tokens over 32768 keys 1830 us whole, 1836 cut after the product; shared tiles
// (32 ragged sequences of up to 60 tokens), whose kernel then spills nothing, 142 and 163. Heads
// of 64 (1592 and 1542) and 256 (over 8192 keys 1054 and 976) keep q whole in sequences of up to
// kPreciseRows rows alone. An fp32 q has more bits than its pieces either way.
template <typename E, int D, int PP>
constexpr bool whole_q() { return sizeof(E) == 2 && (D == 128 || PP > 2); }
template <bool WHOLE>
__device__ __forceinline__ Scaling scaling(const AttnArgs& a) {
    const uint32_t bits = __float_as_uint(a.scale2);
    const bool split = WHOLE && bits >= 0x00800000u;    // has an exponent
    const float q = split ? __uint_as_float(bits & 0x7f800000u) : a.scale2;
    return {a.negate ? -q : q, split ? __uint_as_float((bits & 0x007fffffu) | 0x3f800000u) : 1.f};
}

// ---- products -------------------------------------------------------------------

__device__ __forceinline__ i32x8 operand(const u32x6& v) {
    return (i32x8)__builtin_shufflevector(v, v, 0, 1, 2, 3, 4, 5, -1, -1);
}
__device__ __forceinline__ i32x8 operand(const u32x4& v) {
    return (i32x8)__builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1);
}

// c + entries a (4 bits, unit: byte UA of ua) times pieces b (6 bits, byte UB of ub).
template <int UA, int UB>
__device__ __forceinline__ f32x4 product(const u32x4& a, int ua, const u32x6& b, int ub, f32x4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a), operand(b), c, 4, 2, UA, ua, UB, ub);
}
template <int UA, int UB>
__device__ __forceinline__ f32x16 product(const u32x4& a, int ua, const u32x6& b, int ub, f32x16 c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a), operand(b), c, 4, 2, UA, ua, UB, ub);
}
constexpr int kOne = 0x7f7f7f7f;        // unit 1

// 16 channels' entries of 16 tokens, a channel a lane: lane i of each 16 names the token
// that is to be element i.
__device__ __forceinline__ i32x2 transposed(const char* p) {
    return __builtin_amdgcn_ds_read_tr4_b64_v2i32((__attribute__((address_space(3))) i32x2*)p);
}
__device__ __forceinline__ u32x4 joined(i32x2 a, i32x2 b) {
    return u32x4{(uint32_t)a[0], (uint32_t)a[1], (uint32_t)b[0], (uint32_t)b[1]};
}

// ---- softmax of a lane's 32 scores -------------------------------------------------

// State of a row: the reference m (-inf before its first key), the lane's share of the sum.
// Scores come relative to the reference (0 while there is none). `top` is the largest of
// the row's in the step, over all its lanes. Where scores pass the reference by more than
// kSlack, or there is none yet, it moves: `move(by, factor)` takes `by` from the scores at
// hand and multiplies the output by `factor`.
template <typename F>
__device__ __forceinline__ void follow(float top, float& m, float& l, F move) {
    const bool unset = m == neg_inf();
    if (__builtin_expect(__any(unset ? top > neg_inf() : top > kSlack) != 0, false)) {
        const float by = unset ? (top > neg_inf() ? top : 0.f) : fmaxf(top, 0.f);
        const float factor = unset ? 1.f : __builtin_amdgcn_exp2f(-by);
        if (unset) m = top > neg_inf() ? top : m;
        else m += by;
        l *= factor;
        move(by, factor);
    }
}
__device__ __forceinline__ float reference(float m) { return m == neg_inf() ? 0.f : m; }

// Weights of scores x(i) and the pieces of weights times value scales sv(i); hidden(i) where
// `masked`. Returns the pieces' unit.
template <int PP, typename X, typename SV, typename H>
__device__ __forceinline__ int weights(X x, float& l, SV sv, bool masked, H hidden, u32x6* out) {
    f32x16 lo, hi;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float p = __builtin_amdgcn_exp2f(x(i));
        sum += p;
        if (i < 16) lo[i] = p * sv(i);
        else hi[i - 16] = p * sv(i);
    }
    l += sum;
    if (__builtin_expect(masked, false)) {
        // what is stored behind a hidden key may be anything
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (hidden(i)) {
                if (i < 16) lo[i] = 0.f;
                else hi[i - 16] = 0.f;
            }
    }
    // not negative: compared as integers, in which infinities and NaN come out on top
    int top = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(max(top, __float_as_int(lo[i])), __float_as_int(hi[i]));
    const int e = unit_of<PP>((uint32_t)top);
    split<PP>(lo, hi, e, out);
    return e;
}

__device__ __forceinline__ uint64_t page_row(const CacheArgs& c, uint32_t page, int h) {
    return ((uint64_t)page * c.Hkv + h) << c.shift;
}

// ---------------------------------------------------------------------------
// Few rows (a tile of 16 a sequence and key head, or two): four waves take the work's steps of 128
// keys in turn, each with its own running softmax; they meet in LDS at the end.
//
// v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds operand row (A) or column (B) l % 16,
// k = 32 (l / 16) .. + 31, and of the result column l % 16, rows 4 (l / 16) .. + 3. With
// g = l / 16, n = l % 16:
//   S^T of 16 keys: lane l loads the 32 channels 32 g .. of key n, 16 bytes. Heads of 256
//     take two products; heads of 64 fill k = 64 .. 127 with the same keys again and the
//     next piece of q.
//   O^T of 128 keys: the lane has the weights of keys 16 t + 4 g + i (t < 8, i < 4) of row
//     n; element 2 (4 t + i) is that of t < 4, 2 (4 t + i) + 1 that of t + 4. A value row is
//     put into LDS at the place 32 g + element, from which 16 of them are read transposed.
//
// Bound by memory and by the chains before and after the steps (lengths, table entry, q into
// pieces: 4.7 us; the waves' join; 4.0 to 4.9 for the parts'). One workgroup a compute unit,
// whose waves keep a whole step's keys and values in flight: one token of 32 heads over 8 of
// the keys', 32768 keys of 128 channels, 14.0 us; 32 sequences of 3620 keys 29 (126 MB: 4.3
// TB/s), as much in 1 to 32768 keys each 35, with an fp32 q 39. By two workgroups a compute
// unit, with half the registers, 19.2, 32, 38 and 63. Two tiles at once share what is loaded:
// 6 tokens for each of the ragged sequences 58, by row tiles of 128 rows 70 (calls of 64.5 and
// 76 us; 5 tokens over 32768 keys 28.0 and 28.5).
// ---------------------------------------------------------------------------
constexpr int kStep = 128;

template <int D>
struct FewLds {
    static constexpr int pitch = D / 2 + 16;        // rows read together start in other banks
    char values[kStep * pitch];
    float v_scale[kStep];
    uint8_t k_exp[kStep * (D / 32)];
};

template <typename E, int NP, int PP, int D, int RT>
__device__ __forceinline__ void attend4_few(const Attn4Args& args, const Work& w, int parts, FewLds<D>& lds,
                                            float (*sm)[16 * RT], float (*sl)[16 * RT], float (*so)[16 * RT][D + 4]) {
    const AttnArgs& a = args.a;
    const CacheArgs& c = a.c;
    const Cache4& cache = args.b;
    constexpr int RB = D / 2;                       // bytes of a row
    constexpr int KC = D > 128 ? 2 : 1;             // products of 128 channels
    constexpr int NM = D == 64 ? (NP + 1) / 2 : NP; // products for q's pieces
    constexpr int DT = D / 16;
    constexpr int VL = D / 16;                      // loads of 16 bytes a lane of a step's values
    constexpr bool WHOLE = whole_q<E, D, PP>();
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = lane >> 4, n = lane & 15;

    // Row n of each tile of q, the lane's 32 channels: asked for first, so that cutting them
    // into pieces waits for nothing behind it.
    QBlock<E> qx[RT][KC];
    int pos[RT];
    each<RT>([&](auto r) {
        const int row = w.r0 + 16 * r + n;
        const bool valid = row < w.rows;
        const int tok = valid ? row / a.G : 0;
        const int head = w.h * a.G + (valid ? row - tok * a.G : 0);
        const E* q = static_cast<const E*>(a.q.p) + ((int64_t)(w.first + tok) * a.q.st + head * a.q.sh);
        each<KC>([&](auto cc) { qx[r][cc].load(q + 128 * cc + 32 * (D == 64 ? g & 1 : g), valid); });
        pos[r] = w.p0 + tok;
    });

    // A lane looks up the pages of keys lane and 64 + lane of a step: their rows in the
    // cache's arrays (safe to read in any case), of which every 16th is the first of a tile
    // that lies in one page. Tiles behind the last key are loaded like the others.
    const int32_t* table = c.table + (int64_t)w.b * c.table_stride;
    uint32_t entry[2];
    uint64_t rows[2];
    bool known[2];
    auto load_entries = [&](int t0) {
        entry[0] = page_entry(c, table, t0 + lane);
        entry[1] = page_entry(c, table, t0 + 64 + lane);
    };
    auto find_rows = [&](int t0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int key = t0 + 64 * i + lane;
            rows[i] = page_row(c, page_in(c, entry[i]), w.h) + (key & (c.P - 1));
            known[i] = known_page(c, entry[i], key);
        }
    };
    // byte of the first row of tile t
    auto tile_at = [&](int t) {
        const uint32_t lo = (uint32_t)lane_value((int)(uint32_t)rows[t >> 2], 16 * (t & 3));
        const uint32_t hi = (uint32_t)lane_value((int)(uint32_t)(rows[t >> 2] >> 32), 16 * (t & 3));
        return ((uint64_t)hi << 32 | lo) * RB;
    };
    const uint32_t k_off = n * RB + 16 * (D == 64 ? g & 1 : g);
    u32x4 kr[8][KC];
    uint2 ke[2];
    float vs[2];
    auto load_keys = [&]() {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const uint8_t* p = cache.keys + tile_at(t);
#pragma unroll
            for (int cc = 0; cc < KC; ++cc) kr[t][cc] = *reinterpret_cast<const u32x4*>(p + k_off + 64 * cc);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint8_t* p = cache.k_exp + rows[i] * (D / 32);
            if constexpr (D == 64) ke[i].x = *reinterpret_cast<const uint16_t*>(p);
            else if constexpr (D == 128) ke[i].x = *reinterpret_cast<const uint32_t*>(p);
            else ke[i] = *reinterpret_cast<const uint2*>(p);
            vs[i] = cache.v_scale[rows[i]];
        }
    };
    // piece i of the lane's share of the values: its tile, its row there and the place of
    // that in LDS
    const int v_row = D == 64 ? (lane & 31) >> 1 : D == 128 ? lane >> 2 : lane >> 3;
    const uint32_t v_off = v_row * RB + lane % (D / 32) * 16;
    auto value_place = [&](int i) {
        const int t = D == 64 ? 2 * i + (lane >> 5) : D == 128 ? i : i >> 1, r = D == 256 ? v_row + 8 * (i & 1) : v_row;
        return ((r >> 2) * 32 + 2 * (r & 3) + 8 * (t & 3) + (t >> 2)) * FewLds<D>::pitch + lane % (D / 32) * 16;
    };
    u32x4 vr[VL];
    auto load_values = [&]() {
        each<VL>([&](auto i) {
            uint64_t p = tile_at(D == 64 ? 2 * i : D == 128 ? i : i / 2) + (D == 256 ? i % 2 * 8 * RB : 0);
            if constexpr (D == 64) {
                const uint64_t second = tile_at(2 * i + 1);
                p = lane < 32 ? p : second;
            }
            vr[i] = *reinterpret_cast<const u32x4*>(cache.values + p + v_off);
        });
    };

    int t0 = w.k0 + kStep * wave;
    load_entries(t0);
    __builtin_amdgcn_sched_barrier(0);
    if (t0 < w.k1) {
        find_rows(t0);
        load_keys();
        load_values();
        load_entries(t0 + 4 * kStep);
    }
    __builtin_amdgcn_sched_barrier(0);

    u32x6 qf[RT][KC][NM];
    int qu[RT][KC][2];
    const Scaling by = scaling<WHOLE>(a);
    each<RT>([&](auto r) {
        each<KC>([&](auto cc) {
            if constexpr (D == 64) {
                u32x6 p[NP];
                const int e = qx[r][cc].template split_into<NP>(by.q, p);
                uint32_t u = 0;
                each<NM>([&](auto i) {
                    constexpr int first = 2 * i, second = 2 * i + 1;
#pragma unroll
                    for (int j = 0; j < 6; ++j) {
                        if constexpr (second < NP) qf[r][cc][i][j] = g >> 1 ? p[second][j] : p[first][j];
                        else qf[r][cc][i][j] = g >> 1 ? 0 : p[first][j];
                    }
                    const int at = 2 * i + (g >> 1);
                    u |= (uint32_t)(e == 255 ? 255 : at < NP ? e - 4 * at : 127) << (8 * i);
                });
                qu[r][cc][0] = (int)u;
                qu[r][cc][1] = 0;
            } else {
                const int e = qx[r][cc].template split_into<NP>(by.q, qf[r][cc]);
                units<NP>(e, qu[r][cc]);
            }
        });
    });
    const int p_first = w.p0 + w.r0 / a.G;
    const int p_last = w.p0 + ((w.rows - w.r0 < 16 * RT ? w.rows : w.r0 + 16 * RT) - 1) / a.G;
    f32x4 o[RT][DT];
    float m[RT], l[RT];
    each<RT>([&](auto r) {
#pragma unroll
        for (int i = 0; i < DT; ++i) o[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        m[r] = neg_inf();
        l[r] = 0.f;
    });

    for (; t0 < w.k1; t0 += 4 * kStep) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint8_t* p = lds.k_exp + (64 * i + lane) * (D / 32);
            if constexpr (D == 64) *reinterpret_cast<uint16_t*>(p) = (uint16_t)(known[i] ? ke[i].x : ~0u);
            else if constexpr (D == 128) *reinterpret_cast<uint32_t*>(p) = known[i] ? ke[i].x : ~0u;
            else *reinterpret_cast<uint2*>(p) = known[i] ? ke[i] : make_uint2(~0u, ~0u);
            lds.v_scale[64 * i + lane] = known[i] ? fabsf(vs[i]) : __builtin_nanf("");
        }

        f32x4 s[RT][8];
#pragma unroll
        for (int t = 0; t < 8; ++t)
            each<KC>([&](auto cc) {
                const int ku = lds.k_exp[(16 * t + n) * (D / 32) + (D == 64 ? g & 1 : 4 * cc + g)];
                each<RT>([&](auto r) {
                    if constexpr (cc == 0) {
                        const float ref = WHOLE ? 0.f : -reference(m[r]);
                        s[r][t] = f32x4{ref, ref, ref, ref};
                    }
                    each<NM>([&](auto i) {
                        s[r][t] = product<0, i % 4>(kr[t][cc], ku, qf[r][cc][i], qu[r][cc][i / 4], s[r][t]);
                    });
                });
            });
        each<VL>([&](auto i) { *reinterpret_cast<u32x4*>(lds.values + value_place(i)) = vr[i]; });
        const int tn = t0 + 4 * kStep;
        if (tn < w.k1) {
            find_rows(tn);
            load_keys();
            load_values();
            load_entries(tn + 4 * kStep);
        }

        // a key beyond the row's position or before its window has no weight, whatever is
        // stored there
        const bool masked =
            t0 + kStep - 1 > p_first || t0 + kStep > w.k1 || (a.window > 0 && t0 <= p_last - a.window);
        u32x6 pf[RT][PP];
        int pu[RT][2];
        each<RT>([&](auto r) {
            auto x = [&](int i) { return s[r][i >> 2][i & 3]; };
            if constexpr (WHOLE) {
                const float ref = -reference(m[r]);
#pragma unroll
                for (int i = 0; i < 32; ++i) s[r][i >> 2][i & 3] = __builtin_fmaf(x(i), by.s, ref);
            }
            int up = last_seen(pos[r], t0, w.k1) - 4 * g, dn = before_seen(pos[r], t0, a.window) - 4 * g;
            auto hidden = [&](int i) {
                const int key = 16 * (i >> 2) + (i & 3);
                return key > up || key <= dn;
            };
            if (__builtin_expect(masked, false))
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (hidden(i)) s[r][i >> 2][i & 3] = neg_inf();
            float top = x(0);
#pragma unroll
            for (int i = 1; i < 32; ++i) top = fmaxf(top, x(i));
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = max_halves(top);
            follow(top, m[r], l[r], [&](float by, float factor) {
#pragma unroll
                for (int t = 0; t < 8; ++t) s[r][t] -= by;
#pragma unroll
                for (int i = 0; i < DT; ++i) o[r][i] *= factor;
            });
            asm("" : "+v"(up), "+v"(dn));       // hidden() again: 32 masks kept until then are as many scalars spilled
            float4 sv[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) sv[t] = *reinterpret_cast<const float4*>(&lds.v_scale[16 * t + 4 * g]);
            const int pe = weights<PP>(
                x, l[r], [&](int i) { return (&sv[i >> 2].x)[i & 3]; }, masked, hidden, pf[r]);
            units<PP>(pe, pu[r]);
        });

        const char* at = lds.values + (32 * g + n) * FewLds<D>::pitch;
        each<DT>([&](auto i) {
            const u32x4 v = joined(transposed(at + 8 * i), transposed(at + 16 * FewLds<D>::pitch + 8 * i));
            each<RT>([&](auto r) {
                each<PP>([&](auto p) { o[r][i] = product<0, p % 4>(v, kOne, pf[r][p], pu[r][p / 4], o[r][i]); });
            });
        });
    }
    join_waves<E, D, RT>(late_args(), w, parts, m, l, o, sm, sl, so);
}

template <typename E, int NP, int PP, int D, int RT>
__global__ __launch_bounds__(256, 1) void k_attend4_few(const Attn4Args args) {
    __shared__ float sm[4][16 * RT], sl[4][16 * RT];
    __shared__ __align__(16) float so[4][16 * RT][D + 4];
    __shared__ __align__(16) FewLds<D> lds[4];
    share_work<kUnitCost4, 4 * kStep / kTile>(
        args.a, 16 * RT,
        [&](const Work& w, int parts) {
            attend4_few<E, NP, PP, D, RT>(args, w, parts, lds[threadIdx.x >> 6], sm, sl, so);
        },
        [&](int b) { lose_rows<E, D>(args.a, b, 0, args.a.Hq); });
}

// ---------------------------------------------------------------------------
// Many rows: four waves of 32 rows each share steps of 64 keys, staged in LDS as they lie.
//
// v_mfma_scale_f32_32x32x64_f8f6f4: lane l holds operand row or column l % 32, k = 32 (l /
// 32) .. + 31, and of the result column l % 32, rows 8 (j / 4) + 4 (l / 32) + j % 4, j < 16.
// With half = l / 32:
//   S^T of 32 keys: 64 channels a product, the lane's are 32 (2 c + half) ..
//   O^T of 64 keys: the lane has the weights of keys 8 (j / 4) + 4 half + j % 4 of the first
//     32 (element 2 j) and of the second (2 j + 1). Value rows lie in LDS at the place 32
//     half + element.
//
// Bound by the vector unit and the products' share of its issue slots: exponentials, maxima
// and conversions of 32 scores a lane keep it busy for two thirds of the time, and a scaled
// product takes two to three times the issue cycles of a bf16 one. 4096 tokens of 32 heads
// over 32768 keys 1845 us (heads of 128; 2.06 TFLOP: 1.12 PFLOP/s; 1838 to 1920 from card to
// card), heads of 64 1538; heads of 256 over 8192 keys 973, an fp32 q of heads of 128 859. Tried
// beside it, where it took 1855 (heads of 64 1548): the products of one step's values with the
// next one's scores in one phase 2185; weights as bf16 and values widened in LDS 2115 (heads of
// 64 1484); scores a step ahead by one wave a SIMD 4328, its registers moved to and fro; raised
// priority around the products 1877; workgroups of eight waves, half of them a phase behind, so
// that one half multiplies while the other weighs, 2677 with 128 bytes a lane spilled (heads of
// 64, without spills, 1529).
// ---------------------------------------------------------------------------
template <int D>
struct RowsLds {
    static constexpr int pitch = D / 2 + 16;        // rows read together start in other banks
    char keys[kTile * pitch], values[kTile * pitch];
    float v_scale[kTile];
    uint8_t k_exp[kTile * (D / 32)];
};

template <typename E, int NP, int PP, int D>
__device__ __forceinline__ void attend4_rows(const Attn4Args& args, const Work& w, int parts, RowsLds<D>* lds) {
    const AttnArgs& a = args.a;
    const CacheArgs& c = a.c;
    const Cache4& cache = args.b;
    typedef RowsLds<D> Lds;
    constexpr int RB = D / 2, KC = D / 64, DT = D / 32, pitch = Lds::pitch;
    constexpr int CH = D == 256 ? 2 : 1;            // 16-byte pieces a thread stages of keys, and of values
    constexpr bool WHOLE = whole_q<E, D, PP>();
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int r = w.r0 + 32 * wave + col;
    const bool valid = r < w.rows;
    const int tok = valid ? r / a.G : 0;
    const int head = w.h * a.G + (valid ? r - tok * a.G : 0);
    const int pos = w.p0 + tok;
    const ConstTable table = (ConstTable)(uintptr_t)(c.table + (int64_t)w.b * c.table_stride);

    // Staging: a thread has CH pieces of 16 bytes of the keys and as many of the values
    // (heads of 64: one, in the first two waves of the keys, in the others of the values), a
    // wave the scales of 16 keys. What a wave loads lies in one page (heads of 64: two): page
    // entries and addresses are scalar.
    constexpr int PW = 1024 / RB;                   // keys of a wave's 64 pieces
    const int first_key = D == 64 ? 32 * (wave & 1) : PW * wave;
    const bool takes_keys = D != 64 || wave < 2, takes_values = D != 64 || wave >= 2;
    const uint32_t off = (lane * 16 / RB & 15) * RB + lane * 16 % RB;    // in 16 keys
    int to_k[CH], to_v[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int key = first_key + 4 * PW * i + lane * 16 / RB, m = key & 31, chunk = lane * 16 % RB;
        to_k[i] = key * pitch + chunk;
        to_v[i] = (32 * (m >> 2 & 1) + 2 * (4 * (m >> 3) + (m & 3)) + (key >> 5)) * pitch + chunk;
    }
    u32x4 kr[CH], vr[CH];
    uint2 ke = make_uint2(0, 0);
    float vs = 0.f;
    // page entries of what a wave loads of the step at t0
    struct Entries {
        uint32_t e[2], s;
    };
    auto entries_of = [&](int t0) {
        Entries x;
        x.e[0] = page_entry(c, table, t0 + first_key);
        x.e[1] = D == 128 ? 0 : page_entry(c, table, t0 + first_key + (D == 64 ? 16 : 4 * PW));
        x.s = D == 128 ? x.e[0] : page_entry(c, table, t0 + 16 * wave);
        return x;
    };
    // byte of the first of the 16 keys that key0 of the step at t0 is one of
    auto byte_at = [&](uint32_t e, int t0, int key0) {
        return (page_row(c, page_in(c, e), w.h) + ((t0 + (key0 & ~15)) & (c.P - 1))) * RB;
    };
    auto load = [&](const uint8_t* from, u32x4 (&to)[CH], const Entries& x, int t0) {
        if constexpr (D == 64) {
            const uint64_t b0 = byte_at(x.e[0], t0, first_key), b1 = byte_at(x.e[1], t0, first_key + 16);
            to[0] = *reinterpret_cast<const u32x4*>(from + (lane < 32 ? b0 : b1) + off);
        } else {
            each<CH>([&](auto i) {
                const int key0 = first_key + 4 * PW * i;
                to[i] = *reinterpret_cast<const u32x4*>(from + byte_at(x.e[i], t0, key0) + (key0 & 15) * RB + off);
            });
        }
    };
    auto load_keys = [&](const Entries& x, int t0) {
        if (takes_keys) load(cache.keys, kr, x, t0);
        if (lane < 16) {
            const int t = t0 + 16 * wave;
            const uint64_t row = page_row(c, page_in(c, x.s), w.h) + (t & (c.P - 1));
            const uint8_t* p = cache.k_exp + row * (D / 32) + lane * (D / 32);
            if constexpr (D == 64) ke.x = *reinterpret_cast<const uint16_t*>(p);
            else if constexpr (D == 128) ke.x = *reinterpret_cast<const uint32_t*>(p);
            else ke = *reinterpret_cast<const uint2*>(p);
            vs = fabsf((cache.v_scale + row)[lane]);
            if (!known_page(c, x.s, t)) {
                ke = make_uint2(~0u, ~0u);
                vs = __builtin_nanf("");
            }
        }
    };
    auto load_values = [&](const Entries& x, int t0) {
        if (takes_values) load(cache.values, vr, x, t0);
    };
    auto stage_keys = [&](Lds& to) {
        if (takes_keys) each<CH>([&](auto i) { *reinterpret_cast<u32x4*>(to.keys + to_k[i]) = kr[i]; });
        if (lane < 16) {
            const int key = 16 * wave + lane;
            uint8_t* p = to.k_exp + key * (D / 32);
            if constexpr (D == 64) *reinterpret_cast<uint16_t*>(p) = (uint16_t)ke.x;
            else if constexpr (D == 128) *reinterpret_cast<uint32_t*>(p) = ke.x;
            else *reinterpret_cast<uint2*>(p) = ke;
            to.v_scale[key] = vs;
        }
    };
    auto stage_values = [&](Lds& to) {
        if (takes_values)
            each<CH>([&](auto i) { *reinterpret_cast<u32x4*>(to.values + to_v[i]) = vr[i]; });
    };
    // LDS written by this wave is visible after it; loads stay in flight
    auto step_end = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    Entries next{};                 // of the step that is loaded next
    if (w.k0 < w.k1) {
        next = entries_of(w.k0);
        load_keys(next, w.k0);
        load_values(next, w.k0);
        next = entries_of(w.k0 + kTile);
    }
    u32x6 qf[KC][NP];
    int qu[KC][2];
    const Scaling by = scaling<WHOLE>(a);
    {
        const E* q = static_cast<const E*>(a.q.p) + ((int64_t)(w.first + tok) * a.q.st + head * a.q.sh);
        each<KC>([&](auto cc) {
            QBlock<E> x;
            x.load(q + 64 * cc + 32 * half, valid);
            const int e = x.template split_into<NP>(by.q, qf[cc]);
            units<NP>(e, qu[cc]);
        });
    }
    // positions of this wave's rows
    const int w0 = w.r0 + 32 * wave, w1 = w.rows - w0 < 32 ? w.rows : w0 + 32;
    const int p_first = w.p0 + w0 / a.G, p_last = w.p0 + (w1 - 1) / a.G;

    f32x16 o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] = 0.f;
    float m = neg_inf(), l = 0.f;
    // what scores begin from: minus the reference, as the products' third operand (WHOLE: zero,
    // the reference comes with the rest of the scale)
    f32x16 start;
#pragma unroll
    for (int j = 0; j < 16; ++j) start[j] = 0.f;
    u32x6 pf[PP];           // the step's weights: pieces and their units
    int pu[2];

    auto add_values = [&](const Lds& from) {
        const char* at = from.values + (32 * half + (lane & 15)) * pitch + 8 * (lane >> 4 & 1);
        each<DT>([&](auto i) {
            const u32x4 v = joined(transposed(at + 16 * i), transposed(at + 16 * pitch + 16 * i));
            each<PP>([&](auto p) { o[i] = product<0, p % 4>(v, kOne, pf[p], pu[p / 4], o[i]); });
        });
    };
    f32x16 s[2];
    auto score = [&](const Lds& from) {
        each<2>([&](auto tt) {
            s[tt] = start;
            const int at = 32 * tt + col;
            uint32_t ku[2];
            const uint8_t* p = from.k_exp + at * (D / 32);
            if constexpr (D == 64) ku[0] = *reinterpret_cast<const uint16_t*>(p);
            else ku[0] = *reinterpret_cast<const uint32_t*>(p);
            if constexpr (D == 256) ku[1] = *reinterpret_cast<const uint32_t*>(p + 4);
            // byte 2 c of the lane's words is the unit of block 2 c + half
#pragma unroll
            for (int i = 0; i < (D == 256 ? 2 : 1); ++i) ku[i] >>= 8 * half;
            each<KC>([&](auto cc) {
                const u32x4 k = *reinterpret_cast<const u32x4*>(from.keys + at * pitch + 32 * cc + 16 * half);
                each<NP>([&](auto i) {
                    s[tt] = product<2 * (cc % 2), i % 4>(k, (int)ku[cc / 2], qf[cc][i], qu[cc][i / 4], s[tt]);
                });
            });
        });
    };
    auto weigh = [&](const Lds& from, int t0) {
        auto x = [&](int i) { return s[i >> 4][i & 15]; };
        if constexpr (WHOLE) {
            const float ref = -reference(m);
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i >> 4][i & 15] = __builtin_fmaf(x(i), by.s, ref);
        }
        const bool masked =
            t0 + kTile - 1 > p_first || t0 + kTile > w.k1 || (a.window > 0 && t0 <= p_last - a.window);
        int up = last_seen(pos, t0, w.k1) - 4 * half, dn = before_seen(pos, t0, a.window) - 4 * half;
        auto hidden = [&](int i) {
            const int k = 32 * (i >> 4) + 8 * (i >> 2 & 3) + (i & 3);
            return k > up || k <= dn;
        };
        if (__builtin_expect(masked, false))
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (hidden(i)) s[i >> 4][i & 15] = neg_inf();
        float top = x(0);
#pragma unroll
        for (int i = 1; i < 32; ++i) top = fmaxf(top, x(i));
        top = max_halves(top);
        follow(top, m, l, [&](float by, float factor) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) s[tt] -= by;
#pragma unroll
            for (int i = 0; i < DT; ++i) o[i] *= factor;
            if constexpr (!WHOLE) {
                const float ref = -reference(m);
#pragma unroll
                for (int j = 0; j < 16; ++j) start[j] = ref;
            }
        });
        asm("" : "+v"(up), "+v"(dn));       // hidden() again: 32 masks kept until then are as many scalars spilled
        float4 sv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sv[i] = *reinterpret_cast<const float4*>(from.v_scale + 4 * half + 32 * (i >> 2) + 8 * (i & 3));
        const int pe = weights<PP>(
            x, l, [&](int i) { return (&sv[i >> 2].x)[i & 3]; }, masked, hidden, pf);
        units<PP>(pe, pu);
    };
    if (w.k0 < w.k1) {
        stage_keys(lds[0]);
        stage_values(lds[0]);
        load_keys(next, w.k0 + kTile);
        load_values(next, w.k0 + kTile);
        next = entries_of(w.k0 + 2 * kTile);
        step_end();
    }
    int buf = 0;
    for (int t0 = w.k0; t0 < w.k1; t0 += kTile, buf ^= 1) {
        // nothing to do for rows that see none of the tile's keys
        if (w0 < w1 && t0 <= p_last && (a.window == 0 || (int64_t)t0 + kTile > (int64_t)p_first - a.window + 1)) {
            score(lds[buf]);
            weigh(lds[buf], t0);
            add_values(lds[buf]);
        }
        stage_keys(lds[buf ^ 1]);
        stage_values(lds[buf ^ 1]);
        load_keys(next, t0 + 2 * kTile);
        load_values(next, t0 + 2 * kTile);
        next = entries_of(t0 + 3 * kTile);
        step_end();
    }

    l += __shfl_xor(l, 32, 64);
    if (!valid) return;
    const AttnArgs z = late_args();
    const int64_t row = (int64_t)(w.first + tok) * z.Hq + head;
    const bool seen = row_sees(pos, z.window, w.k0, w.k1);
    const float inv = parts == 1 ? row_inverse(l, seen) : 1.f;
    const int64_t part = row * z.splits + w.part;
    E* out = static_cast<E*>(z.out.p) + ((int64_t)(w.first + tok) * z.out.st + head * z.out.sh);
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int d = 32 * i + 8 * q + 4 * half;
            const float v[4] = {o[i][4 * q] * inv, o[i][4 * q + 1] * inv, o[i][4 * q + 2] * inv, o[i][4 * q + 3] * inv};
            if (parts == 1) store4(out + d, v);
            else store4(z.part_o + part * D + d, v);
        }
    if (half != 0) return;
    if (parts > 1) z.part_ml[part] = make_float2(m, l == 0.f && seen ? -1.f : l);
    else if (z.lse) z.lse[row] = row_lse(m, l, seen);
    if (z.splits > 1 && w.part == 0) z.parts[row] = parts;
}

// SHARED: in equal shares (share_work), else a workgroup for each row tile, head and range
// of keys (find_work). Sequences of few rows beside ones of many keep their weights to
// three pieces.
template <typename E, int NP, int PP, int D, bool SHARED>
__global__ __launch_bounds__(256, few_held(D, sizeof(E) == 4)) void k_attend4_rows(const Attn4Args args) {
    __shared__ __align__(16) RowsLds<D> lds[2];
    auto attend = [&](const Work& w, int parts) {
        if constexpr (PP == 2)
            if (w.rows <= kPreciseRows) return attend4_rows<E, NP, 3, D>(args, w, parts, lds);
        attend4_rows<E, NP, PP, D>(args, w, parts, lds);
    };
    if constexpr (SHARED) {
        share_work<kTileCost4>(
            args.a, 128,
            [&](const Work& w, int parts) {
                __syncthreads();        // the work before has been read from LDS
                attend(w, parts);
            },
            [&](int b) { lose_rows<E, D>(args.a, b, 0, args.a.Hq); });
    } else {
        Work w;
        auto lost = [&](int b, int h) { lose_rows<E, D>(args.a, b, h * args.a.G, (h + 1) * args.a.G); };
        if (find_work(args.a, 128, w, lost)) attend(w, args.a.splits);
    }
}

template <typename E, int NP, int PP, int D>
hipError_t launch_rows(const Attn4Args& a, const AttnPlan& plan, hipStream_t s) {
    if (plan.shared) {
        k_attend4_rows<E, NP, PP, D, true><<<dim3((unsigned)plan.blocks), 256, 0, s>>>(a);
        return hipGetLastError();
    }
    return launch_in_pieces(plan.blocks, [&](uint32_t first, unsigned n) {
        Attn4Args piece = a;
        piece.a.first_block = first;
        k_attend4_rows<E, NP, PP, D, false><<<n, 256, 0, s>>>(piece);
    });
}

template <typename E, int D>
hipError_t launch(const Attn4Args& a, const AttnPlan& plan, hipStream_t s) {
    constexpr bool wide = sizeof(E) == 4;
    hipError_t e = hipSuccess;
    if (plan.few) {
        k_attend4_few<E, wide ? 5 : 4, wide ? 5 : 3, D, 1><<<dim3((unsigned)plan.blocks), 256, 0, s>>>(a);
        e = hipGetLastError();
    } else if (plan.pair) {
        if constexpr (D <= 128)
            k_attend4_few<E, wide ? 5 : 4, wide ? 5 : 3, D, 2><<<dim3((unsigned)plan.blocks), 256, 0, s>>>(a);
        e = hipGetLastError();
    } else {
        e = launch_rows<E, wide ? 5 : 4, wide ? 5 : 2, D>(a, plan, s);
    }
    return e != hipSuccess ? e : launch_join<E, D>(a.a, plan, s);
}

template <typename E>
hipError_t launch_dim(const Attn4Args& a, const AttnPlan& plan, hipStream_t s) {
    switch (a.a.c.D) {
        case 64: return launch<E, 64>(a, plan, s);
        case 128: return launch<E, 128>(a, plan, s);
        default: return launch<E, 256>(a, plan, s);
    }
}

}  // namespace

hipError_t launch_cache4_attention(const CacheArgs& c, const Cache4& b, const AttnPlan& plan, const Heads& q, int Hq,
                                   float scale, int window, const Heads& out, float* lse, void* ws, hipStream_t s) {
    const Attn4Args a{attn_args(c, plan, q, Hq, scale, window, out, lse, ws), b};
    return c.dt == Dt::BF16 ? launch_dim<uint16_t>(a, plan, s) : launch_dim<float>(a, plan, s);
}

}  // namespace sffn
