// Attention of new tokens over the paged 8-bit cache.
//
//   s_j = scale q . (k8_j sk_j),  o = sum_j p_j (v8_j sv_j) / sum_j p_j,  p_j = exp(s_j - max)
//
// One pass over the keys with the running maximum m and sum l of the softmax.
// Entries are small integers, exact in bf16, so q . k8 on the bf16 matrix
// cores (fp32 accumulation) loses nothing; the page's scale multiplies the
// fp32 score, and the value's scale the weight p before it is rounded to bf16
// (p sv, so that a page of small values keeps its relative precision). An fp32
// q is taken as three bf16 pieces (24 bits), and so are the weights. For a bf16 q
// the weights are two pieces (16 bits) where a sequence has up to kPreciseRows rows
// a key head, and one (up to 2^-8 of each weight, as much as the result's own rounding)
// above, where the second costs a third: 4096 tokens over 32768 keys 1.81 ms, with
// two pieces 2.39; heads of 64 1.25 and 1.62; heads of 256 over 8192 keys 0.91 and
// 1.18. A sequence's own tokens decide it, not the call's: what else is in the batch
// does not change how exact a row is.
//
// Both kernels compute S^T = K Q^T and O^T = V^T P^T, which keeps a query row
// in one matrix column: the lane that holds scores of a row holds that row's
// weights in just the order in which the second product wants them, provided
// the key a lane's matrix row stands for is chosen for it. So P never leaves
// the registers, the softmax needs one or two lane exchanges a tile, and the
// cache keeps its values transposed ([D][token]) to be that product's operand
// as they lie.
#include <type_traits>

#include "attn_work.hpp"

namespace sffn {

namespace {

// Four int8 as bf16 (exact).
__device__ __forceinline__ uint2 widen4(uint32_t from) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float x = (float)(int8_t)(from >> (16 * i));
        const float y = (float)(int8_t)(from >> (16 * i + 8));
        w[i] = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
    }
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
    const uint2 a = widen4(lo), b = widen4(hi);
    return __builtin_bit_cast(bf16x8, make_uint4(a.x, a.y, b.x, b.y));
}

// Eight fp32 as NP bf16 pieces: their sum is x to 8 NP bits.
template <int NP>
__device__ __forceinline__ void pieces(const float* x, bf16x8* out) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = x[i];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = round2(r[2 * i], r[2 * i + 1]);
            if (p + 1 < NP) {
                r[2 * i] -= bf16_lo(w[i]);
                r[2 * i + 1] -= bf16_hi(w[i]);
            }
        }
        out[p] = __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
    }
}

// x by a power of two (exact, unless it leaves bf16's range), 0 or what is not finite.
__device__ __forceinline__ bf16x8 times(bf16x8 x, float by) {
    const uint4 w = __builtin_bit_cast(uint4, x);
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = round2(bf16_lo(in[i]) * by, bf16_hi(in[i]) * by);
    return __builtin_bit_cast(bf16x8, make_uint4(out[0], out[1], out[2], out[3]));
}

template <typename E, int NP>
__device__ __forceinline__ void load_q(const E* p, bool valid, bool negate, bf16x8* out) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (valid) Elem<E>::load8(p, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = negate ? -x[i] : x[i];
    pieces<NP>(x, out);
}

// ---------------------------------------------------------------------------
// Few rows (a tile of 16, or two: single tokens, drafts): memory-bound, each key
// and value is read once. Four waves take the split's 64-key steps in turn, each with its
// own running softmax, straight from memory into matrix operands; they meet in
// LDS at the end. The values of a step and the keys of the next are in flight while
// it computes: 16 KB a wave of heads of 128, 33 MB over the chip, which its memory
// needs to stream. One token over 32768 keys of 8 heads of 128 (67 MB): 19.2 us, of
// which 13 are the bytes at a copy's rate; 32 ragged sequences (237 MB): 57 us, 4.2
// TB/s; with an fp32 q 22 and 82 (one workgroup a compute unit).
//
// v_mfma_f32_16x16x32_bf16: lane l holds operand row (A) or column (B) l % 16,
// k = 8 (l / 16) .. + 7, and of the result column l % 16, rows 4 (l / 16) ..
// + 3. With g = l / 16:
//   S^T: step (c, u) takes d = 64 c + 16 g + 8 u .. + 7, so a lane's 16-byte
//     load of a key is two steps' operand. Matrix row m of score tile t (of
//     four) stands for key 16 (m / 4) + 4 t + m % 4, so that lane l gets keys
//     16 g + 4 t + i (i < 4) of query row l % 16: sixteen consecutive ones.
//   O^T: step u takes keys 16 g + 8 u .. + 7: the weights are in place, and a
//     lane's 16-byte load of a value row [d][16 g ..] is two steps' operand.
// ---------------------------------------------------------------------------
template <typename E, int NP, int PP, int D, int RT>
__device__ __forceinline__ void attend_few(const AttnArgs& a, const Work& w, int parts, float (*sm)[16 * RT],
                                           float (*sl)[16 * RT], float (*so)[16 * RT][D + 4]) {
    constexpr int KC = D / 64, DT = D / 16;
    const CacheArgs& c = a.c;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = lane >> 4, n = lane & 15, gk = n >> 2;
    int pos[RT];            // of the lane's row in each tile of 16

    const uint32_t head_bytes = (uint32_t)c.P * D;      // of one page
    const uint32_t page_bytes = c.Hkv * head_bytes;
    const int32_t* table = c.table + (int64_t)w.b * c.table_stride;
    const int8_t* keys = c.keys + (size_t)w.h * head_bytes + (((16 * gk) & (c.P - 1)) + (n & 3)) * D + 16 * g;
    const int8_t* values = c.values + (size_t)w.h * head_bytes + n * c.P + ((16 * g) & (c.P - 1));
    const float *k_scale = c.k_scale + w.h, *v_scale = c.v_scale + w.h;
    uint4 kr[4][KC];
    auto load_keys = [&](uint32_t entry, int t0) {
        const int8_t* p = keys + (uint64_t)page_in(c, entry) * page_bytes + (t0 & (c.P - 1)) * D;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int cc = 0; cc < KC; ++cc) kr[t][cc] = *reinterpret_cast<const uint4*>(p + 4 * t * D + 64 * cc);
    };

    int t0 = w.k0 + kTile * wave;
    uint32_t entry_k = page_entry(c, table, t0 + 16 * gk), entry_v = page_entry(c, table, t0 + 16 * g);
    if (t0 < w.k1) load_keys(entry_k, t0);

    bf16x8 qf[RT][KC][2][NP];
    f32x4 o[RT][DT];
    float m[RT], l[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int row = w.r0 + 16 * r + n;
        const bool valid = row < w.rows;
        const int tok = valid ? row / a.G : 0;
        const int head = w.h * a.G + (valid ? row - tok * a.G : 0);
        const E* q = static_cast<const E*>(a.q.p) + ((int64_t)(w.first + tok) * a.q.st + head * a.q.sh);
#pragma unroll
        for (int cc = 0; cc < KC; ++cc)
#pragma unroll
            for (int u = 0; u < 2; ++u) load_q<E, NP>(q + 64 * cc + 16 * g + 8 * u, valid, a.negate, qf[r][cc][u]);
#pragma unroll
        for (int i = 0; i < DT; ++i) o[r][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        pos[r] = w.p0 + tok;
        m[r] = neg_inf();
        l[r] = 0.f;
    }
    const int p_first = w.p0 + w.r0 / a.G;
    const int p_last = w.p0 + ((w.rows - w.r0 < 16 * RT ? w.rows : w.r0 + 16 * RT) - 1) / a.G;

    for (; t0 < w.k1; t0 += 4 * kTile) {
        // values and scales of this step, page ids of the next
        uint4 vr[DT];
        const uint32_t page = page_in(c, entry_v);
        const int8_t* vp = values + (uint64_t)page * page_bytes + (t0 & (c.P - 1));
#pragma unroll
        for (int i = 0; i < DT; ++i) vr[i] = *reinterpret_cast<const uint4*>(vp + 16 * i * c.P);
        float ks = k_scale[(size_t)page * c.Hkv], vs = v_scale[(size_t)page * c.Hkv];
        const bool known = known_page(c, entry_v, t0 + 16 * g);
        const int tn = t0 + 4 * kTile;
        entry_k = page_entry(c, table, tn + 16 * gk);
        entry_v = page_entry(c, table, tn + 16 * g);

        f32x4 s[RT][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int r = 0; r < RT; ++r) s[r][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int cc = 0; cc < KC; ++cc)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const bf16x8 kf = u ? widen(kr[t][cc].z, kr[t][cc].w) : widen(kr[t][cc].x, kr[t][cc].y);
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int p = 0; p < NP; ++p)
                            s[r][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[r][cc][u][p], s[r][t], 0, 0, 0);
                }
        }
        if (tn < w.k1) load_keys(entry_k, tn);

        ks = known ? ks * a.scale2 : __builtin_nanf("");
        vs = known ? vs : __builtin_nanf("");
        bf16x8 pf[RT][2][PP];
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float x[16], pvs = vs;
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] = s[r][e >> 2][e & 3] * ks;
            // a key beyond the row's position or before its window has no weight,
            // whatever is stored there: a select, and a scale of 0 where the row
            // sees none of the lane's sixteen (they share a page)
            if (t0 + kTile - 1 > p_first || t0 + kTile > w.k1 || (a.window > 0 && t0 <= p_last - a.window)) {
                const int up = last_seen(pos[r], t0, w.k1) - 16 * g, dn = before_seen(pos[r], t0, a.window) - 16 * g;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e > up || e <= dn) x[e] = neg_inf();
                if (up < 0 || dn >= 15) pvs = 0.f;
            }
            float top = x[0];
#pragma unroll
            for (int e = 1; e < 16; ++e) top = fmaxf(top, x[e]);
            top = fmaxf(top, __shfl_xor(top, 16, 64));
            top = max_halves(top);
            if (__any(top > m[r] + kSlack)) {
                const float to = fmaxf(m[r], top);
                const float alpha = __builtin_amdgcn_exp2f(m[r] - (to == neg_inf() ? 0.f : to));
                m[r] = to;
                l[r] *= alpha;
#pragma unroll
                for (int i = 0; i < DT; ++i) o[r][i] *= alpha;
            }
            const float ref = m[r] == neg_inf() ? 0.f : m[r];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float pv[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float p = __builtin_amdgcn_exp2f(x[8 * u + e] - ref);
                    l[r] += p;
                    pv[e] = p * pvs;
                }
                pieces<PP>(pv, pf[r][u]);
            }
        }
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bf16x8 vf = u ? widen(vr[i].z, vr[i].w) : widen(vr[i].x, vr[i].y);
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int p = 0; p < PP; ++p)
                        o[r][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pf[r][u][p], o[r][i], 0, 0, 0);
            }
    }

    join_waves<E, D, RT>(a, w, parts, m, l, o, sm, sl, so);
}

template <typename E, int NP, int PP, int D, int RT>
__global__ __launch_bounds__(256, few_held(D, NP == 3)) void k_attend_few(const AttnArgs a) {
    __shared__ float sm[4][16 * RT], sl[4][16 * RT];
    __shared__ __align__(16) float so[4][16 * RT][D + 4];
    share_work(
        a, 16 * RT, [&](const Work& w, int parts) { attend_few<E, NP, PP, D, RT>(a, w, parts, sm, sl, so); },
        [&](int b) { lose_rows<E, D>(a, b, 0, a.Hq); });
}

// ---------------------------------------------------------------------------
// Many rows (chunks of a prompt): NW waves of 32 rows each share 64-key steps,
// widened to bf16 once for all of them on the way into LDS. Rows run over
// (token, head of the group), so every head that shares the keys shares the tile.
//
// A step of a wave is two phases of about equal length: M(t), the matrix
// products O += P(t - 1) V(t - 1) and S = K(t) Q with this thread's share of
// widening later tiles in their shadow, and V(t), the softmax of S. With eight
// waves the second four (the second wave of every SIMD) run one phase behind, so
// that one wave of a SIMD keeps the matrix cores busy while the other computes
// weights; barriers between phases hold them there. Counting phases, K(t) is
// read in 2t and 2t + 1, V(t) in 2t + 2 and 2t + 3, the scales of t in 2t + 1 and
// 2t + 2; the first four waves write their part of K(t + 1) and V(t) in phase 2t,
// the others theirs in 2t + 1, and one wave the scales of t in its phase V(t - 1),
// 2t (2t - 1 where there are four waves): always after the last read of what the
// (double) buffer held and before its first use.
//
// Bound by the matrix cores and by power: a step of eight waves takes 3620 cycles
// of which the matrix cores are busy for 2050, and what shortens it lowers the
// clock (1.8 to 2.1 GHz; with a cache of zeros, which costs less power, a version
// of 1.92 ms took 1.63). A chunk of 4096 tokens over 32768 keys, 32 heads of 128:
// 1.89 ms (median; least 1.81), 1.09 PF, 79% of what a library's product of 16384^3
// reaches.
//
// What a wave loads lies in one page, so page entries and addresses are scalar.
//
// v_mfma_f32_32x32x16_bf16: lane l holds operand row or column l % 32, k = 8
// (l / 32) .. + 7, and of the result column l % 32, rows 8 (i / 4) + 4 (l / 32)
// + i % 4, i < 16. With half = l / 32, matrix row m of a 32-key score tile
// stands for key 16 ((m / 4) % 2) + 4 (m / 8) + m % 4, so that lane l holds
// keys 16 half + i: what the second product's steps u = 0, 1 take as k.
//
// LDS: keys [64][D] in matrix-row order and values [D][64], bf16, rows padded by
// 16 bytes: a read's sixteen consecutive rows then start in other banks (68 and
// 36 words apart), and every address of a step is one lane's base and a constant.
// ---------------------------------------------------------------------------
template <typename E, int NP, int PP, int D, int NW>
__device__ __forceinline__ void attend_rows(const AttnArgs& a, const Work& w, int parts, char* lds,
                                            float4 (*scales)[4]) {
    constexpr int NT = 64 * NW, KS = D / 16, DT = D / 32;
    constexpr int CH = (4 * D + NT - 1) / NT;           // 16-byte pieces a thread loads of keys, and of values
    constexpr int KP = 2 * D + 16, VP = 2 * kTile + 16; // row pitches in bytes
    constexpr int KB = kTile * KP, BUF = KB + D * VP;   // bytes of the keys, of one buffer
    const CacheArgs& c = a.c;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int r = w.r0 + 32 * wave + col;
    const bool valid = r < w.rows;
    const int tok = valid ? r / a.G : 0;
    const int head = w.h * a.G + (valid ? r - tok * a.G : 0);
    const int pos = w.p0 + tok;

    // Staging: wave part i of this wave, (wave + i NW) of the tile's D / 16, is 64
    // pieces of 16 bytes of the keys (token-major) and of the values (16 keys of
    // a channel, channels first), all of the same 16 keys.
    const uint32_t head_bytes = (uint32_t)c.P * D;      // of one page
    const uint32_t page_bytes = c.Hkv * head_bytes;
    const ConstTable table = (ConstTable)(uintptr_t)(c.table + (int64_t)w.b * c.table_stride);
    const int8_t* keys = c.keys + (size_t)w.h * head_bytes;
    const int8_t* values = c.values + (size_t)w.h * head_bytes;
    uint32_t off_k[CH], off_v[CH];      // in the page; P = 128 adds 64 tokens for its second half
    int to_k[CH], to_v[CH];             // in LDS
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int p = tid + i * NT, key = p / (D / 16) & 63, piece = p % (D / 16), d = p % D, g = p / D & 3;
        off_k[i] = (key & (c.P - 1)) * D + 16 * piece;
        off_v[i] = d * c.P + ((16 * g) & (c.P - 1));
        to_k[i] = ((key & 32) | (key & 12) << 1 | (key & 16) >> 2 | (key & 3)) * KP + 32 * piece;
        to_v[i] = KB + d * VP + 32 * g;
    }
    auto active = [&](int i) { return 4 * D % NT == 0 || (wave + i * NW) * 64 < 4 * D; };
    uint4 kr[CH], vr[CH];
    uint32_t entry_k[CH], entry_v[CH], entry_s = 0;
    float ks_in = 0.f, vs_in = 0.f;
    bool known = false;
    // t0: first key of the tile (tiles past the last one load what is never used)
    auto key_pages = [&](int t0) {
#pragma unroll
        for (int i = 0; i < CH; ++i) entry_k[i] = page_entry(c, table, t0 + 16 * ((wave + i * NW) * 64 / D & 3));
    };
    auto value_pages = [&](int t0) {
#pragma unroll
        for (int i = 0; i < CH; ++i) entry_v[i] = page_entry(c, table, t0 + 16 * ((wave + i * NW) * 64 / D & 3));
    };
    const bool scaler = wave == (NW == 8 ? 4 : 0) && lane < 4;
    auto scale_pages = [&](int t0) {
        if (scaler) entry_s = page_entry(c, c.table + (int64_t)w.b * c.table_stride, t0 + 16 * lane);
    };
    auto load_keys = [&](int i, int t0) {
        if (active(i))
            kr[i] = *reinterpret_cast<const uint4*>(keys + (uint64_t)page_in(c, entry_k[i]) * page_bytes +
                                                    (t0 & (c.P - 1)) * D + off_k[i]);
    };
    auto load_values = [&](int i, int t0) {
        if (active(i))
            vr[i] = *reinterpret_cast<const uint4*>(values + (uint64_t)page_in(c, entry_v[i]) * page_bytes +
                                                    (t0 & (c.P - 1)) + off_v[i]);
    };
    auto load_scales = [&](int t0) {
        if (scaler) {
            const size_t srow = (size_t)page_in(c, entry_s) * c.Hkv + w.h;
            ks_in = c.k_scale[srow];
            vs_in = c.v_scale[srow];
            known = known_page(c, entry_s, t0 + 16 * lane);
        }
    };
    auto stage_keys = [&](int i, int buf) {
        if (active(i)) {
            char* to = lds + buf * BUF + to_k[i];
            *reinterpret_cast<bf16x8*>(to) = widen(kr[i].x, kr[i].y);
            *reinterpret_cast<bf16x8*>(to + 16) = widen(kr[i].z, kr[i].w);
        }
    };
    auto stage_scales = [&](int buf) {
        if (scaler) {
            const float ks = known ? ks_in * a.scale2 : __builtin_nanf(""), vs = known ? vs_in : __builtin_nanf("");
            // of each 16 keys: the key scale (with the softmax's), and of the value
            // scale the logarithm (base 2) and the reciprocal of one factor, and the
            // other factor. The first goes into the exponent, so it may not take
            // weights that count to where fp32 ends: scales far from 1 are a mantissa
            // and a power of two there, all others themselves and 1. What is not finite
            // is the other factor: the sum of the weights does not know the values.
            float first = vs, rest = 1.f;
            if (!(vs >= 0x1p-64f && vs <= 0x1p100f)) {
                const bool finite = vs > 0.f && vs < __builtin_huge_valf();
                first = finite ? 2.f * __builtin_amdgcn_frexp_mantf(vs) : 1.f;
                rest = finite ? __builtin_amdgcn_ldexpf(1.f, __builtin_amdgcn_frexp_expf(vs) - 1) : vs;
            }
            scales[buf][lane] = make_float4(ks, __builtin_amdgcn_logf(first), __builtin_amdgcn_rcpf(first), rest);
        }
    };
    // LDS written by this wave is visible after it; loads stay in flight
    auto phase_end = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };

    const bool late = NW == 8 && wave >= 4;
    // One of the 8 CH words (four entries) of a thread's share of the keys of the
    // step after the one at t0 and of that step's values: to bf16, every second one
    // into LDS with the one before it, the last of a piece followed by the load of
    // the piece's next.
    uint4 wide;
    auto stage_word = [&](int i, int buf, int t0) {
        const int piece = i / 4 % CH, part = i & 3;
        if (!active(piece)) return;
        const bool is_key = i < 4 * CH;
        const uint4& from = is_key ? kr[piece] : vr[piece];
        const uint2 v = widen4(part == 0 ? from.x : part == 1 ? from.y : part == 2 ? from.z : from.w);
        if (part & 1) {
            wide.z = v.x;
            wide.w = v.y;
            char* to = lds + (is_key ? (buf ^ 1) * BUF + to_k[piece] : buf * BUF + to_v[piece]);
            *reinterpret_cast<uint4*>(to + 16 * (part >> 1)) = wide;
        } else {
            wide.x = v.x;
            wide.y = v.y;
        }
        if (part == 3) {
            if (is_key) load_keys(piece, t0 + 2 * kTile);
            else load_values(piece, t0 + kTile);
        }
    };
    // the scales of the step after the one at t0
    auto next_scales = [&](int buf, int t0) {
        stage_scales(buf);
        load_scales(t0 + 2 * kTile);
        scale_pages(t0 + 3 * kTile);
    };
    if (w.k0 < w.k1) {
        key_pages(w.k0);
        value_pages(w.k0);
        scale_pages(w.k0);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            load_keys(i, w.k0);
            load_values(i, w.k0);
        }
        load_scales(w.k0);
        key_pages(w.k0 + kTile);
        value_pages(w.k0 + kTile);
        scale_pages(w.k0 + kTile);
    }
    bf16x8 qf[KS][NP];
    {
        const E* q = static_cast<const E*>(a.q.p) + ((int64_t)(w.first + tok) * a.q.st + head * a.q.sh);
#pragma unroll
        for (int s = 0; s < KS; ++s) load_q<E, NP>(q + 16 * s + 8 * half, valid, a.negate, qf[s]);
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

    bf16x8 pf[2][2][PP];
    f32x16 s[2];
    // Phase M of the step at t0: O += P V of the tile before (in buffer `buf` ^ 1;
    // not in the first step), S = K Q of this one and the staging (not in what
    // follows the last step). The products go in groups of two (64 cycles): before
    // each the operands of the next group are read from LDS, and each takes its part
    // of the staging, a word at a time: six instructions, which fit the issue slots
    // that the products leave free. (Pieces of four words held the products up:
    // phase M took 1840 cycles instead of 1500, the chunk above 1845 us instead of
    // 1830; in phase V the staging took longer still, 1885 to 2090 us. Groups of four
    // take 1% more.) The phase has priority over the softmax of the SIMD's other
    // wave: a product that starts late is lost, a weight is not (without: 4% more).
    //
    // The scales are phase V's work: their chain of loads, logarithm and store
    // delayed every wave by 250 cycles in phase M (1920 us instead of 1845). Where a
    // SIMD has one wave they come last there, behind the arithmetic that needs no
    // load (heads of 256, 4096 tokens over 8192 keys: 922 us instead of 1076).
    auto phase_m = [&](auto with_values, auto with_keys, int buf, int t0) {
        constexpr int NV = with_values.value ? 4 * DT : 0, NK = with_keys.value ? 2 * KS : 0, N = NV + NK;
        constexpr int GS = 2, NG = N / GS;
        const char* vb = lds + (buf ^ 1) * BUF + KB + col * VP + 32 * half;
        const char* kb = lds + buf * BUF + col * KP + 16 * half;
        auto read = [&](int i) {
            // values: (tile half, step, channel tile); keys: (16 channels, tile half)
            const char* p = i < NV ? vb + i % DT * 32 * VP + 64 * (i / (2 * DT)) + 16 * (i / DT % 2)
                                   : kb + (i - NV) % 2 * 32 * KP + 32 * ((i - NV) / 2);
            return *reinterpret_cast<const bf16x8*>(p);
        };
        bf16x8 f[2][GS];
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < GS; ++i) f[0][i] = read(i);
        if (with_keys.value)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int j = 0; j < 16; ++j) s[tt][j] = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            if (g + 1 < NG)
#pragma unroll
                for (int i = 0; i < GS; ++i) f[(g + 1) & 1][i] = read((g + 1) * GS + i);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < GS; ++j) {
                const int i = g * GS + j;
                if (i < NV) {
#pragma unroll
                    for (int p = 0; p < PP; ++p)
                        o[i % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            f[g & 1][j], pf[i / (2 * DT)][i / DT % 2][p], o[i % DT], 0, 0, 0);
                } else {
                    const int tt = (i - NV) % 2, k = (i - NV) / 2;
#pragma unroll
                    for (int p = 0; p < NP; ++p)
                        s[tt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[g & 1][j], qf[k][p], s[tt], 0, 0, 0);
                }
            }
            if (with_keys.value)
#pragma unroll
                for (int i = 0; i < 8 * CH; ++i)
                    if (g == i * NG / (8 * CH)) stage_word(i, buf, t0);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (with_keys.value) {
            key_pages(t0 + 3 * kTile);
            value_pages(t0 + 2 * kTile);
        }
        __builtin_amdgcn_s_setprio(0);
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    if (w.k0 < w.k1) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            stage_keys(i, 0);
            load_keys(i, w.k0 + kTile);
        }
        key_pages(w.k0 + 2 * kTile);
        if (NW == 4) next_scales(0, w.k0 - kTile);
        phase_end();
        if (late) {
            next_scales(0, w.k0 - kTile);
            phase_end();
        }
    }
    // Phase V of the step at t0. A wave whose rows see none of the tile's keys
    // goes through it like the others (all keys are hidden): few tiles of a row
    // tile are such, and every wave meets every barrier.
    auto phase_v = [&](int buf, int t0) {
        if (NW == 8) next_scales(buf ^ 1, t0);
        // the value scale (its first factor) goes into the exponent, p vs =
        // 2^(x + log2 vs), and comes out of the sum of each 16 keys again
        float4 f[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) f[tt] = scales[buf][2 * tt + half];
        if (t0 + kTile - 1 > p_first || t0 + kTile > w.k1 || (a.window > 0 && t0 <= p_last - a.window)) {
            // as in k_attend_few: hidden keys by a select, and no scales
            // where the row sees none of the lane's sixteen
            const int up = last_seen(pos, t0, w.k1) - 16 * half, dn = before_seen(pos, t0, a.window) - 16 * half;
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int key = 32 * tt + j;
                    s[tt][j] = key > up || key <= dn ? neg_inf() : s[tt][j] * f[tt].x;
                }
                f[tt].x = 1.f;
                if (32 * tt > up || 32 * tt + 15 <= dn) f[tt] = make_float4(1.f, 0.f, 0.f, 1.f);
            }
        }
        float top[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            top[tt] = s[tt][0];
#pragma unroll
            for (int j = 1; j < 16; ++j) top[tt] = fmaxf(top[tt], s[tt][j]);
        }
        float most = fmaxf(top[0] * f[0].x, top[1] * f[1].x);
        most = max_halves(most);
        if (__any(most > m + kSlack)) {
            const float to = fmaxf(m, most);
            const float alpha = __builtin_amdgcn_exp2f(m - (to == neg_inf() ? 0.f : to));
            m = to;
            l *= alpha;
#pragma unroll
            for (int i = 0; i < DT; ++i) o[i] *= alpha;
        }
        const float ref = m == neg_inf() ? 0.f : m;
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const float shift = f[tt].y - ref;
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float pv[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    pv[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[tt][8 * u + e], f[tt].x, shift));
                    sum += pv[e];
                }
                pieces<PP>(pv, pf[tt][u]);
            }
            l += sum * f[tt].z;
        }
        if (__any(f[0].w != 1.f || f[1].w != 1.f)) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int p = 0; p < PP; ++p) pf[tt][u][p] = times(pf[tt][u][p], f[tt].w);
        }
        if (NW == 4) next_scales(buf ^ 1, t0);
    };
    if (w.k0 < w.k1) {
        phase_m(no, yes, 0, w.k0);
        phase_end();
        phase_v(0, w.k0);
        phase_end();
        int buf = 1;
        for (int t0 = w.k0 + kTile; t0 < w.k1; t0 += kTile, buf ^= 1) {
            phase_m(yes, yes, buf, t0);
            phase_end();
            phase_v(buf, t0);
            phase_end();
        }
        if (NW == 8 && !late) phase_end();
        phase_m(yes, no, buf, w.k1);
    }

    l += __shfl_xor(l, 32, 64);
    if (!valid) return;
    const int64_t row = (int64_t)(w.first + tok) * a.Hq + head;
    const bool seen = row_sees(pos, a.window, w.k0, w.k1);
    const float inv = parts == 1 ? row_inverse(l, seen) : 1.f;
    const int64_t part = row * a.splits + w.part;
    E* out = static_cast<E*>(a.out.p) + ((int64_t)(w.first + tok) * a.out.st + head * a.out.sh);
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int d = 32 * i + 8 * q + 4 * half;
            const float v[4] = {o[i][4 * q] * inv, o[i][4 * q + 1] * inv, o[i][4 * q + 2] * inv, o[i][4 * q + 3] * inv};
            if (parts == 1) store4(out + d, v);
            else store4(a.part_o + part * D + d, v);
        }
    if (half != 0) return;
    if (parts > 1) a.part_ml[part] = make_float2(m, l == 0.f && seen ? -1.f : l);
    else if (a.lse) a.lse[row] = row_lse(m, l, seen);
    if (a.splits > 1 && w.part == 0) a.parts[row] = parts;
}

// SHARED: in equal shares (share_work), else a workgroup for each row tile, head and
// range of keys (find_work).
template <typename E, int NP, int PP, int D, int NW, bool SHARED>
__global__ __launch_bounds__(64 * NW, NW == 8 || D == 256 || NP == 3 ? 1 : 2) void k_attend_rows(const AttnArgs a) {
    __shared__ __align__(16) char lds[2 * (kTile * (2 * D + 16) + D * (2 * kTile + 16))];
    __shared__ float4 scales[2][4];
    // PP 1: sequences of few rows beside ones of many keep their weights to two pieces
    // (2048 tokens over 32768 keys beside 31 single tokens: 1.86 ms, with one 1.68)
    auto attend = [&](const Work& w, int parts) {
        if constexpr (PP == 1)
            if (w.rows <= kPreciseRows) return attend_rows<E, NP, 2, D, NW>(a, w, parts, lds, scales);
        attend_rows<E, NP, PP, D, NW>(a, w, parts, lds, scales);
    };
    if constexpr (SHARED) {
        share_work(
            a, 32 * NW,
            [&](const Work& w, int parts) {
                __syncthreads();        // the work before has been read from LDS
                attend(w, parts);
            },
            [&](int b) { lose_rows<E, D>(a, b, 0, a.Hq); });
    } else {
        Work w;
        auto lost = [&](int b, int h) { lose_rows<E, D>(a, b, h * a.G, (h + 1) * a.G); };
        if (find_work(a, 32 * NW, w, lost)) attend(w, a.splits);
    }
}

template <typename E, int NP, int PP, int D, int NW>
hipError_t launch_rows(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
    if (plan.shared) {
        k_attend_rows<E, NP, PP, D, NW, true><<<dim3((unsigned)plan.blocks), 64 * NW, 0, s>>>(a);
        return hipGetLastError();
    }
    return launch_in_pieces(plan.blocks, [&](uint32_t first, unsigned n) {
        AttnArgs piece = a;
        piece.first_block = first;
        k_attend_rows<E, NP, PP, D, NW, false><<<n, 64 * NW, 0, s>>>(piece);
    });
}

template <typename E, int NP, int D>
hipError_t launch(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
    const dim3 grid((unsigned)plan.blocks);
    hipError_t e = hipSuccess;
    if (plan.few) {
        k_attend_few<E, NP, NP == 1 ? 2 : 3, D, 1><<<grid, 256, 0, s>>>(a);
    } else if (plan.pair) {
        if constexpr (D <= 128) k_attend_few<E, NP, NP == 1 ? 2 : 3, D, 2><<<grid, 256, 0, s>>>(a);
    } else if constexpr (NP == 3) {
        e = launch_rows<E, 3, 3, D, 4>(a, plan, s);
    } else if (plan.pieces == 2) {
        e = launch_rows<E, 1, 2, D, 4>(a, plan, s);
    } else {
        e = launch_rows<E, 1, 1, D, D <= 128 ? 8 : 4>(a, plan, s);
    }
    if (e == hipSuccess) e = hipGetLastError();
    return e != hipSuccess ? e : launch_join<E, D>(a, plan, s);
}

template <typename E, int NP>
hipError_t launch_dim(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
    switch (a.c.D) {
        case 64: return launch<E, NP, 64>(a, plan, s);
        case 128: return launch<E, NP, 128>(a, plan, s);
        default: return launch<E, NP, 256>(a, plan, s);
    }
}

}  // namespace

hipError_t launch_cache_attention(const CacheArgs& c, const AttnPlan& plan, const Heads& q, int Hq, float scale,
                                  int window, const Heads& out, float* lse, void* ws, hipStream_t s) {
    const AttnArgs a = attn_args(c, plan, q, Hq, scale, window, out, lse, ws);
    return c.dt == Dt::BF16 ? launch_dim<uint16_t, 1>(a, plan, s) : launch_dim<float, 3>(a, plan, s);
}

}  // namespace sffn
