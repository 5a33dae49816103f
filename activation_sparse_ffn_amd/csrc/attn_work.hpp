// What the attention kernels share, whatever the cache holds: the sequences, rows and keys
// of a workgroup's work, the softmax's reference, and the join of parts.
#pragma once

#include <math.h>

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

// EXTRA, ROUND: of kernels whose beginnings and ends hide behind no other's work. A unit then
// costs EXTRA more than its steps; with a ROUND, where every unit can begin a share of its
// own, shares are multiples of ROUND steps (what a workgroup takes at a time) and long enough
// for that if there are twice as many workgroups as units. (4-bit cache: 32 sequences of 1 to 32768 keys, single tokens, 35 us with EXTRA
// 16 and 65 with 0; 6 tokens each 58 and 114; one sequence takes the same.)
template <int EXTRA = 0, int ROUND = 1, typename F, typename L>
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
        return (steps > kLeast ? steps : kLeast) + EXTRA;
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
    const int units_of_all = B <= 64 ? lane_value(wave_scan(x.units, add), 63) : 0;
    if (B <= 64 && units_of_all <= (int)gridDim.x && total < 1 << 29) {
        const int unrounded = x.cost, shared = share;
        auto round_up = [&](int to) {
            round_to = share = to;
            sum_costs(x);
            return lane_value(x.cost, 63);
        };
        int rounded;
        if constexpr (EXTRA == 0 || ROUND == 1) {
            rounded = round_up(share);
        } else {
            // (at least one step: a call whose sequences have no new tokens has no share of 0)
            const int steps_alone = total - EXTRA * units_of_all, grid = (int)gridDim.x;
            const int alone = steps_alone > 0 ? steps_alone : 1;
            auto whole = [&](int n) {
                int to = ((alone + n - 1) / n + ROUND - 1) / ROUND * ROUND;
                if (a.splits > 1 && to < longest / (a.splits - 1) + 1) to = longest / (a.splits - 1) + 1;
                return to;
            };
            rounded = round_up(whole(grid));
            if (rounded / share > grid && 2 * units_of_all <= grid) rounded = round_up(whole(grid - units_of_all));
        }
        if (rounded / share > (int)gridDim.x) {
            round_to = 0;
            share = shared;
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

// The four waves of a few-row workgroup have each taken some of the keys of its 16 RT
// rows: lane l holds of row 16 r + l % 16 the channels 16 i + 4 (l / 16) .. + 3 of the
// output in o[r][i], the reference m[r], and its own share of the sum l[r]. They meet in
// LDS; the result goes out, or to the workspace as one of the rows' parts.
template <typename E, int D, int RT>
__device__ __forceinline__ void join_waves(const AttnArgs& a, const Work& w, int parts, float (&m)[RT], float (&l)[RT],
                                           f32x4 (&o)[RT][D / 16], float (*sm)[16 * RT], float (*sl)[16 * RT],
                                           float (*so)[16 * RT][D + 4]) {
    constexpr int DT = D / 16;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = lane >> 4, n = lane & 15;
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

// The join of a plan's parts, where it has more than one.
template <typename E, int D>
hipError_t launch_join(const AttnArgs& a, const AttnPlan& plan, hipStream_t s) {
    if (plan.splits == 1) return hipSuccess;
    const int64_t rows = a.c.T * a.Hq;      // half a million at most, for two parts each (kPartBytes)
    if (rows < kWaveRows) k_attend_join<E, D, 256><<<dim3((unsigned)rows), 256, 0, s>>>(a);
    else k_attend_join<E, D, 64><<<dim3((unsigned)((rows + 3) / 4)), 256, 0, s>>>(a);
    return hipGetLastError();
}

inline AttnArgs attn_args(const CacheArgs& c, const AttnPlan& plan, const Heads& q, int Hq, float scale, int window,
                          const Heads& out, float* lse, void* ws) {
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
    return a;
}

}  // namespace

}  // namespace sffn
