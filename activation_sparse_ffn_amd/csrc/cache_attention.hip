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
#include <math.h>

#include <type_traits>

#include "attn_common.hpp"
#include "attn_launch.hpp"

namespace sffn {

namespace {

constexpr int kTile = 64;           // keys of one step
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

struct AttnArgs {
    CacheArgs c;
    Heads q, out;
    int Hq, G, window, splits;
    int chunk, row_tiles;
    uint32_t first_block;   // of this launch, where a call's workgroups take several
    float scale2;           // |scale| log2 e; a negative scale turns q round
    bool negate;
    float* lse;             // [T, Hq] or null
    float* part_o;          // [T Hq, splits, D], unnormalised
    int* parts;             // [T Hq]: parts of each row (few rows: as many as its keys' shares)
    float2* part_ml;        // [T Hq, splits]: reference maximum (base 2), sum; see row_inverse
};

__device__ __forceinline__ float neg_inf() { return -__builtin_huge_valf(); }

// v of lane l, the same in every lane
__device__ __forceinline__ int lane_value(int v, int l) { return __builtin_amdgcn_readlane(v, l); }

// The new tokens of a sequence. Positions fit 31 bits (the host bounds the
// table's capacity and the call's tokens).
struct Sequence {
    int first;              // first token of the sequence's in the call
    int p0;                 // position of that token
    int64_t rows;           // (token, head) rows of the sequence and a key head
};

// False when the sequence has no new tokens.
__device__ __forceinline__ bool find_sequence(const AttnArgs& a, int b, Sequence& q) {
    const CacheArgs& c = a.c;
    int last = b + 1;
    q.first = b;
    if (c.cu) {
        q.first = c.cu[b];
        last = c.cu[b + 1];
    }
    if (q.first < 0 || last > c.T || last <= q.first) return false;
    const int n = last - q.first, capacity = c.max_pages << c.shift;
    int L = c.lens[b];
    if (L < 0) L = 0;
    // more tokens than the table has room for: every row sees one of no page
    if (L > capacity) L = capacity + n;
    q.p0 = L - n;
    q.rows = (int64_t)(n < c.max_new ? n : c.max_new) * a.G;
    return true;
}

// Keys [lo, hi) that rows r0 .. r1 - 1 of a sequence see, lo a multiple of kTile.
__device__ __forceinline__ void keys_seen(const AttnArgs& a, const Sequence& q, int r0, int r1, int& lo, int& hi) {
    hi = q.p0 + (r1 - 1) / a.G + 1;
    lo = 0;
    if (a.window > 0) {
        const int64_t from = (int64_t)q.p0 + r0 / a.G - a.window + 1;
        if (from > 0) lo = (int)from / kTile * kTile;
    }
    if (hi < lo) hi = lo;
}

// NaN in the rows that lost_tokens names, heads h0 .. h1 - 1, by the whole workgroup.
template <typename E, int D>
__device__ __forceinline__ void lose_rows(const AttnArgs& a, int b, int h0, int h1) {
    int from, to;
    if (!lost_tokens(a.c, b, from, to)) return;
    const float nan = __builtin_nanf(""), none[4] = {nan, nan, nan, nan};
    const int64_t n = (int64_t)(to - from) * (h1 - h0) * (D / 4);
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
        const int64_t r = i / (D / 4), t = from + r / (h1 - h0);
        const int h = h0 + (int)(r % (h1 - h0)), d = 4 * (int)(i % (D / 4));
        store4(static_cast<E*>(a.out.p) + (t * a.out.st + h * a.out.sh) + d, none);
        if (a.lse && d == 0) a.lse[t * a.Hq + h] = nan;
    }
}

// The rows and keys of one piece of work.
struct Work {
    int first, p0;          // as in Sequence
    int rows;
    int r0;                 // first row of this tile
    int k0, k1;             // keys
    int b, h;
    int part;               // of the rows' parts
};

// Work of a workgroup of k_attend_rows: a row tile and a range of a.chunk keys.
// False when the tile has no rows. `lost(b, h)` is called by one workgroup for each
// sequence and key head.
template <typename F>
__device__ __forceinline__ bool find_work(const AttnArgs& a, int tile_rows, Work& w, F lost) {
    const CacheArgs& c = a.c;
    uint32_t id = a.first_block + blockIdx.x;
    // Workgroup i runs on XCD i % 8: heads stay with their XCD's cache where there
    // are eight of them.
    w.h = (int)(id % (uint32_t)c.Hkv);
    id /= (uint32_t)c.Hkv;
    int tile;
    if (c.B <= 64) {
        // the longest sequences first, and of each the longest rows: what begins
        // last is short. (With the sequences taking turns a chunk of 1500 tokens
        // over 6001 keys among five shorter ones took 303 us.)
        w.part = (int)(id % (uint32_t)a.splits);
        id /= (uint32_t)a.splits;
        tile = a.row_tiles - 1 - (int)(id % (uint32_t)a.row_tiles);
        const int place = (int)(id / (uint32_t)a.row_tiles);
        const int lane = threadIdx.x & 63;
        const int length = lane < c.B ? c.lens[lane] : 0;
        int before = 0;
        for (int j = 0; j < c.B; ++j) {
            const int other = lane_value(length, j);
            before += other > length || (other == length && j < lane);
        }
        w.b = __ffsll((unsigned long long)__ballot(lane < c.B && before == place)) - 1;
    } else {
        const uint32_t turn = id % (uint32_t)c.B;
        id /= (uint32_t)c.B;
        w.part = (int)(id % (uint32_t)a.splits);
        id /= (uint32_t)a.splits;
        tile = a.row_tiles - 1 - (int)id;
        // the sequences change places from tile to tile, so that a long one among
        // short ones does not fall to some XCDs alone
        w.b = (int)((turn + (uint32_t)tile) % (uint32_t)c.B);
    }
    if (tile == 0 && w.part == 0) lost(w.b, w.h);
    Sequence q;
    if (!find_sequence(a, w.b, q)) return false;
    const int64_t r0 = (int64_t)tile * tile_rows;
    if (r0 >= q.rows) return false;
    w.first = q.first;
    w.p0 = q.p0;
    w.rows = (int)q.rows;
    w.r0 = (int)r0;
    int lo, hi;
    keys_seen(a, q, w.r0, w.rows - w.r0 < tile_rows ? w.rows : w.r0 + tile_rows, lo, hi);
    const int64_t k0 = lo + (int64_t)w.part * a.chunk;
    w.k0 = (int)(k0 < hi ? k0 : hi);
    w.k1 = w.part == a.splits - 1 || hi < k0 + a.chunk ? hi : (int)k0 + a.chunk;
    return true;
}

// Sum (or largest, of values >= 0) of lanes 0 .. l, in lane l: within rows of 16
// lanes, then across them.
template <typename Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false));   // row_shr:1
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false));   // row_shr:2
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false));   // row_shr:4
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false));   // row_shr:8
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false));   // row_bcast:15
    return op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false));    // row_bcast:31
}

// The work of all sequences, row tiles and heads in a row, cut into equal shares of
// the grid's workgroups (as many as the chip holds at once): lengths are known on the
// device alone, and a grid for the longest would be nearly all empty for ragged
// ones (32 sequences of 1 .. 32768 keys, one token each, took 86 us so, 55.6 in even
// shares; finer ranges cost more in empty workgroups than they gave; 6 tokens of 4
// heads each in coarse ranges 477, in shares 74). In steps of 64
// keys, a unit (row tile and head) costs as many as the sequence's longest tile, but
// at least kLeast: what beginning and ending one takes. Units of at most kLeast
// steps, or all where nothing joins parts, go whole to the workgroup in whose share
// they begin. Where there are workgroups enough, every unit begins a share of its own
// (cost rounded up to shares), so that no workgroup has the end of one and the
// beginning of the next one after another. A workgroup looks at all lengths twice, 64
// at a time: nothing for 64 sequences, but 1024 of 1 to 200 keys take 124 us (64 of
// them 10.6), 1024 of 1 to 4096 310 + 16 (200 at a copy's rate), and the state of the
// walk costs every kernel that shares 47 to 82 spilled scalars. `work(w, parts)` is called for each piece
// of the workgroup's; a row whose part 0 it is has `parts` parts in all. `lost(b)` is
// called by one workgroup for each sequence with tokens that are not computed.
constexpr int kLeast = 8;

template <typename F, typename L>
__device__ __forceinline__ void share_work(const AttnArgs& a, int tile_rows, F work, L lost) {
    const int lane = threadIdx.x & 63;
    const int B = a.c.B, Hkv = a.c.Hkv;
    // 64 sequences from b0 on, one a lane: where they are, their units, a unit's steps
    // and the cost of them up to the lane's. (The host has seen to it that the cost of
    // all fits 31 bits.)
    struct Lane {
        Sequence q;
        int units, steps, cost;
    };
    int round_to = 0;           // 0: costs as they are, else rounded up to multiples of it
    auto padded = [&](int steps) {
        if (round_to > 0) return (steps + round_to - 1) / round_to * round_to;
        return steps > kLeast ? steps : kLeast;
    };
    auto add = [](int p, int q) { return p + q; };
    auto sum_costs = [&](Lane& y) { y.cost = wave_scan(padded(y.steps) * y.units, add); };
    auto look = [&](int b0) {
        Lane y;
        y.units = 0;
        y.steps = 1;
        if (b0 + lane < B && find_sequence(a, b0 + lane, y.q)) {
            const int rows = (int)y.q.rows, tiles = (rows + tile_rows - 1) / tile_rows;
            int lo, hi;
            keys_seen(a, y.q, tiles == 1 ? 0 : (tiles - 1) * tile_rows, rows, lo, hi);
            if (tiles > 1 && a.window > 0) {
                // any tile's: the window and the tile's tokens, from a multiple of 64 on
                const int64_t most = (int64_t)a.window + tile_rows / a.G + 2 + kTile;
                lo = 0;
                if (hi > most) hi = (int)most;
            }
            y.steps = hi - lo > kTile ? (hi - lo + kTile - 1) / kTile : 1;
            y.units = tiles * Hkv;
        }
        sum_costs(y);
        return y;
    };
    auto longest_of = [&](const Lane& y) {
        return lane_value(wave_scan(y.units > 0 ? y.steps : 0, [](int p, int q) { return p > q ? p : q; }), 63);
    };
    auto look_for_lost = [&](int b0) {
        int from, to;
        uint64_t found = __ballot(b0 + lane < B && lost_tokens(a.c, b0 + lane, from, to));
        for (; found != 0; found &= found - 1) {
            const uint32_t b = b0 + __ffsll((unsigned long long)found) - 1;
            if (b % gridDim.x == blockIdx.x) lost((int)b);
        }
    };
    Lane x = look(0);
    look_for_lost(0);
    int total = lane_value(x.cost, 63), longest = longest_of(x);
    for (int b0 = 64; b0 < B; b0 += 64) {
        const Lane y = look(b0);
        look_for_lost(b0);
        const int l = longest_of(y);
        total += lane_value(y.cost, 63);
        longest = l > longest ? l : longest;
    }
    int share = (total + (int)gridDim.x - 1) / (int)gridDim.x;
    if (share < kLeast) share = kLeast;
    // no more parts than the workspace has room for
    if (a.splits > 1 && share < longest / (a.splits - 1) + 1) share = longest / (a.splits - 1) + 1;
    if (B <= 64 && lane_value(wave_scan(x.units, add), 63) <= (int)gridDim.x && total < 1 << 29) {
        round_to = share;
        const int unrounded = x.cost;
        sum_costs(x);
        const int rounded = lane_value(x.cost, 63);
        if (rounded / share > (int)gridDim.x) {
            round_to = 0;
            x.cost = unrounded;
        } else {
            total = rounded;
        }
    }
    if ((int64_t)blockIdx.x * share >= total) return;
    const int c0 = (int)blockIdx.x * share, c1 = total - c0 > share ? c0 + share : total;

    // the sequence in whose cost c0 lies
    int start = 0, b0 = 0;                  // start: cost before the 64, then before the unit
    while (start + lane_value(x.cost, 63) <= c0) {
        start += lane_value(x.cost, 63);
        b0 += 64;
        x = look(b0);
    }
    int at = __ffsll((unsigned long long)__ballot(start + x.cost > c0)) - 1;
    int steps = lane_value(x.steps, at), units = lane_value(x.units, at);
    start += lane_value(x.cost, at) - padded(steps) * units;
    int unit = (c0 - start) / padded(steps);
    start += unit * padded(steps);
    while (start < c1) {
        int from = 0, to = steps, part = 0, parts = 1;
        if (a.splits == 1 || steps <= kLeast) {
            if (start < c0) to = 0;         // another workgroup's
        } else {
            if (start < c0) {
                from = c0 - start;
                part = (c0 - start + share - 1) / share;
                parts = part + 1;           // more than one: that is all the others have to know
            }
            if (c1 - start < steps) {
                to = c1 - start;
                parts = part + 2 + (steps - 1 - to) / share;
            }
        }
        if (from < to) {
            Work w;
            Sequence q;
            w.first = q.first = lane_value(x.q.first, at);
            w.p0 = q.p0 = lane_value(x.q.p0, at);
            w.rows = lane_value((int)x.q.rows, at);
            q.rows = w.rows;
            const int tile = unit / Hkv;
            w.h = unit - tile * Hkv;
            w.r0 = tile * tile_rows;
            w.b = b0 + at;
            w.part = part;
            int lo, hi;
            keys_seen(a, q, w.r0, w.rows - w.r0 < tile_rows ? w.rows : w.r0 + tile_rows, lo, hi);
            // a tile of fewer steps than the longest has none in the first ones
            const int none = steps - (hi - lo > kTile ? (hi - lo + kTile - 1) / kTile : 1);
            w.k0 = lo + (from > none ? from - none : 0) * kTile;
            w.k1 = to == steps ? hi : lo + (to > none ? to - none : 0) * kTile;
            work(w, parts);
        }
        start += padded(steps);
        if (++unit < units) continue;
        unit = 0;
        do {
            if (b0 + ++at >= B) return;
            if (at == 64) {
                at = 0;
                b0 += 64;
                x = look(b0);
            }
            units = lane_value(x.units, at);
        } while (units == 0);
        steps = lane_value(x.steps, at);
    }
}

// The table's entry for the page of position `pos` (the last one behind the
// table's end). It is loaded a step before it is used and checked only then, so
// that nothing waits for it: known_page says whether it names a page of the
// pool, page_in one that is safe to read in any case (a row that sees a key of
// an unknown page gets its NaN from the scales).
typedef const __attribute__((address_space(4))) int32_t* ConstTable;    // read by scalar loads
template <typename Row>
__device__ __forceinline__ uint32_t page_entry(const CacheArgs& c, Row row, int pos) {
    const int idx = pos >> c.shift;
    return (uint32_t)row[idx < c.max_pages ? idx : c.max_pages - 1];
}
__device__ __forceinline__ bool known_page(const CacheArgs& c, uint32_t entry, int pos) {
    return entry < (uint32_t)c.n_pages && (pos >> c.shift) < c.max_pages;
}
__device__ __forceinline__ uint32_t page_in(const CacheArgs& c, uint32_t entry) {
    return entry < (uint32_t)c.n_pages ? entry : (uint32_t)c.n_pages - 1;
}

// Larger of the two halves' values, in every lane.
__device__ __forceinline__ float max_halves(float v) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Whether the row at position p sees a key of [k0, k1).
__device__ __forceinline__ bool row_sees(int p, int window, int k0, int k1) {
    const int from = window > 0 && p - (window - 1) > k0 ? p - (window - 1) : k0;
    return from <= p && from < k1;
}

// The last of the first `keys` keys from t0 on that a row at position p sees,
// and the last one before those it sees, both relative to t0.
__device__ __forceinline__ int last_seen(int p, int t0, int k1) { return (p < k1 - 1 ? p : k1 - 1) - t0; }
__device__ __forceinline__ int before_seen(int p, int t0, int window) {
    if (window == 0) return -1;
    const int64_t d = (int64_t)p - window - t0;
    return d < -1 ? -1 : (int)d;
}

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

// The running maximum m is a reference, not always the largest score: it moves
// (and the sums are scaled) only when a row's scores pass it by more than
// kSlack, which spares nearly every step the products over the whole output
// tile. Weights then reach 2^kSlack, nothing to fp32 sums or to bf16's range.
constexpr float kSlack = 8.f;

// How much a part with reference m and sum l counts where the common one is M.
// A part without finite scores has m = -inf: it counts nothing, unless a NaN
// was among its scores.
__device__ __forceinline__ float part_factor(float m, float l, float M) {
    if (m == neg_inf()) return l != l ? 1.f : 0.f;
    return __builtin_amdgcn_exp2f(m - M);
}

// 1 / l of a row's final sum. A row that saw keys (seen) with nothing but -inf
// scores has no softmax: NaN; one that saw none gives zeros.
__device__ __forceinline__ float row_inverse(float l, bool seen) {
    if (l == 0.f) return seen ? __builtin_nanf("") : 0.f;
    return 1.f / l;
}
__device__ __forceinline__ float row_lse(float M, float l, bool seen) {
    if (l == 0.f) return seen ? __builtin_nanf("") : neg_inf();
    return (M + __log2f(l)) * kLn2;
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

    __syncthreads();        // the work before has been read from LDS
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        l[r] += __shfl_xor(l[r], 16, 64);
        l[r] += __shfl_xor(l[r], 32, 64);
        if (g == 0) {
            sm[wave][16 * r + n] = m[r];
            sl[wave][16 * r + n] = l[r];
        }
#pragma unroll
        for (int i = 0; i < DT; ++i) *reinterpret_cast<f32x4*>(&so[wave][16 * r + n][16 * i + 4 * g]) = o[r][i];
    }
    __syncthreads();

    // thread: row n2 of each tile of 16, D / 16 consecutive channels
    const int d0 = (threadIdx.x & 15) * (D / 16);
#pragma unroll 1
    for (int n2 = threadIdx.x >> 4; n2 < 16 * RT; n2 += 16) {
        const int r2 = w.r0 + n2;
        if (r2 >= w.rows) return;
        float M = neg_inf(), sum = 0.f, f[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) M = fmaxf(M, sm[v][n2]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            f[v] = part_factor(sm[v][n2], sl[v][n2], M);
            sum += f[v] * sl[v][n2];
        }
        float acc[D / 16];
#pragma unroll
        for (int d = 0; d < D / 16; ++d) acc[d] = 0.f;
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (f[v] != 0.f)
#pragma unroll
                for (int d = 0; d < D / 16; ++d) acc[d] += f[v] * so[v][n2][d0 + d];
        const int tok2 = r2 / a.G, head2 = w.h * a.G + r2 - tok2 * a.G;
        const int64_t row = (int64_t)(w.first + tok2) * a.Hq + head2;
        const bool seen = row_sees(w.p0 + tok2, a.window, w.k0, w.k1);
        if (parts == 1) {
            const float inv = row_inverse(sum, seen);
            E* out = static_cast<E*>(a.out.p) + ((int64_t)(w.first + tok2) * a.out.st + head2 * a.out.sh) + d0;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) acc[d] *= inv;
#pragma unroll
            for (int d = 0; d < D / 16; d += 4) store4(out + d, acc + d);
            if (a.lse && d0 == 0) a.lse[row] = row_lse(M, sum, seen);
        } else {
            const int64_t part = row * a.splits + w.part;
#pragma unroll
            for (int d = 0; d < D / 16; d += 4) store4(a.part_o + part * D + d0 + d, acc + d);
            if (d0 == 0) a.part_ml[part] = make_float2(M, sum == 0.f && seen ? -1.f : sum);
        }
        if (a.splits > 1 && w.part == 0 && d0 == 0) a.parts[row] = parts;
    }
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

// ---------------------------------------------------------------------------
// Joins the parts of a row: NT threads, each with four channels of every SG-th part
// (four loads in flight); the SG sums meet in LDS or by lane exchanges, in a fixed
// order. A workgroup takes one row: 4.5 us for 32 rows of 64 parts, launch and a chain
// of two loads. From kWaveRows rows on, which have few parts each, a wave does: 32768
// rows 15 us (as workgroups 45), 8192 9.4 (14.2); 1024 rows of up to 66 parts would
// take 11.1 (8.7). A sum of -1 marks a part whose keys were seen but all scored -inf.
// Tokens of no sequence, or beyond its first max_new, have no parts and are left
// alone.
// ---------------------------------------------------------------------------
constexpr int64_t kWaveRows = 4096;
template <typename E, int D, int NT>
__global__ __launch_bounds__(256) void k_attend_join(const AttnArgs a) {
    constexpr int CG = D / 4, SG = NT / CG, IN = 4;
    const int lane = threadIdx.x & 63, tid = threadIdx.x % NT;
    const int64_t row64 = (int64_t)blockIdx.x * (256 / NT) + threadIdx.x / NT;
    if (row64 >= a.c.T * a.Hq) return;
    const int row = (int)row64, t = row / a.Hq;
    // loaded before it is known whether the row has parts
    const float2* ml = a.part_ml + (int64_t)row * a.splits;
    const int parts = a.parts[row];
    const float2 mine = lane < a.splits ? ml[lane] : make_float2(0.f, 0.f);
    if (a.c.cu) {
        int lo = 0, hi = a.c.B;             // cu[lo] <= t < cu[hi], where t is in a sequence
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (a.c.cu[mid] <= t) lo = mid;
            else hi = mid;
        }
        const int first = a.c.cu[lo], last = a.c.cu[hi];
        if (first < 0 || last > a.c.T || t < first || t >= last || t - first >= a.c.max_new) return;
    }
    if (parts == 1) return;     // written at once
    const int cg = tid % CG, sg = tid / CG;
    const float4* o = reinterpret_cast<const float4*>(a.part_o + (int64_t)row * a.splits * D) + cg;
    float4 v[IN];
    auto load = [&](int s) {
#pragma unroll
        for (int i = 0; i < IN; ++i)
            if (s + i * SG < parts) v[i] = o[(int64_t)(s + i * SG) * CG];
    };
    load(sg);                   // in flight during the sums over the parts

    float M = lane < parts ? mine.x : neg_inf();
    for (int s = lane + 64; s < parts; s += 64) M = fmaxf(M, ml[s].x);
#pragma unroll
    for (int w = 32; w >= 1; w >>= 1) M = fmaxf(M, __shfl_xor(M, w, 64));
    float sum = 0.f, marks = 0.f;
    for (int s = lane; s < parts; s += 64) {
        const float2 p = s == lane ? mine : ml[s];
        const float f = part_factor(p.x, p.y, M);
        if (f != 0.f) sum += f * p.y;
        else if (p.y < 0.f) marks = 1.f;
    }
    sum = wave_sum(sum);
    marks = wave_sum(marks);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = sg; s < parts; s += IN * SG) {
        if (s != sg) load(s);
#pragma unroll
        for (int i = 0; i < IN; ++i) {
            if (s + i * SG >= parts) break;
            const float2 p = ml[s + i * SG];
            const float f = part_factor(p.x, p.y, M);
            if (f == 0.f) continue;         // what counts nothing may hold anything
            acc.x += f * v[i].x;
            acc.y += f * v[i].y;
            acc.z += f * v[i].z;
            acc.w += f * v[i].w;
        }
    }
    float r[4] = {acc.x, acc.y, acc.z, acc.w};
    if constexpr (NT == 64) {
#pragma unroll
        for (int w = 32; w >= CG; w >>= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] += __shfl_xor(r[i], w, 64);
    } else {
        __shared__ float4 so[SG][CG];
        so[sg][cg] = acc;
        __syncthreads();
        r[0] = r[1] = r[2] = r[3] = 0.f;
        if (sg == 0)
#pragma unroll
            for (int i = 0; i < SG; ++i) {
                const float4 p = so[i][cg];
                r[0] += p.x;
                r[1] += p.y;
                r[2] += p.z;
                r[3] += p.w;
            }
    }
    const int h = row - t * a.Hq;
    const float inv = row_inverse(sum, marks != 0.f);
    if (sg == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] *= inv;
        store4(static_cast<E*>(a.out.p) + ((int64_t)t * a.out.st + h * a.out.sh) + 4 * cg, r);
    }
    if (a.lse && tid == 0) a.lse[row] = row_lse(M, sum, marks != 0.f);
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
    if (e != hipSuccess || plan.splits == 1) return e;
    const int64_t rows = a.c.T * a.Hq;      // half a million at most, for two parts each (kPartBytes)
    if (rows < kWaveRows) k_attend_join<E, D, 256><<<dim3((unsigned)rows), 256, 0, s>>>(a);
    else k_attend_join<E, D, 64><<<dim3((unsigned)((rows + 3) / 4)), 256, 0, s>>>(a);
    return hipGetLastError();
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
    AttnArgs a{};
    a.c = c;
    a.q = q;
    a.out = out;
    a.Hq = Hq;
    a.G = Hq / c.Hkv;
    a.window = window;
    a.splits = plan.splits;
    a.chunk = (int)plan.chunk;
    a.row_tiles = (int)plan.row_tiles;
    a.scale2 = fabsf(scale) * kLog2e;
    a.negate = scale < 0.f;
    a.lse = lse;
    if (plan.splits > 1) {
        const size_t rows = (size_t)c.T * Hq;
        a.part_o = static_cast<float*>(ws);
        a.part_ml = reinterpret_cast<float2*>(a.part_o + rows * plan.splits * c.D);
        a.parts = reinterpret_cast<int*>(a.part_ml + rows * plan.splits);
    }
    return c.dt == Dt::BF16 ? launch_dim<uint16_t, 1>(a, plan, s) : launch_dim<float, 3>(a, plan, s);
}

}  // namespace sffn
