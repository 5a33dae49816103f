// Host-side launchers of the attention-side operators. Each returns the
// hipGetLastError() of its launches; callers have validated every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch.hpp"

namespace sffn {

// HIP takes fewer than 2^32 threads in a grid. Larger ones (of workgroups of up to
// 512) are launched in pieces: launch(first, blocks) for each.
constexpr int64_t kMostBlocks = (int64_t)1 << 22;
template <typename F>
inline hipError_t launch_in_pieces(int64_t blocks, F launch) {
    for (int64_t first = 0; first < blocks; first += kMostBlocks) {
        launch((uint32_t)first, (unsigned)(blocks - first < kMostBlocks ? blocks - first : kMostBlocks));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// A [T, heads, head_dim] view (strides in elements).
struct Heads {
    void* p;
    int64_t st, sh;
};

// ---- head norms and rotary positions ----------------------------------------
struct RopeArgs {
    Dt dt;
    int n_q, n_k, D, R, max_pos;    // R: rotated elements of each head
    bool interleaved, norm;
    float eps;
    int64_t T;
    Heads q, k;                     // forward: inputs; backward: the forward's inputs
    Heads g_q, g_k;                 // backward: gradients of the outputs
    Heads q_out, k_out;             // forward: outputs; backward: gradients of the inputs
    const int32_t* pos;             // [T]
    const float* table;             // [max_pos, R]: cos | sin
    const void *q_w, *k_w;          // [D] or null (ones)
    float *g_qw, *g_kw;             // backward: [D] fp32 or null
    float* partial;                 // backward with norm: rope_partial_floats(...)
};
size_t rope_partial_floats(const RopeArgs& a);
hipError_t launch_rope(const RopeArgs& a, hipStream_t s);
hipError_t launch_rope_backward(const RopeArgs& a, hipStream_t s);

// ---- 8-bit cache ----------------------------------------------------------------
struct CacheArgs {
    int8_t *keys, *values;          // [n_pages, Hkv, P, D], [n_pages, Hkv, D, P]
    float *k_scale, *v_scale;       // [n_pages, Hkv]
    int64_t n_pages;
    int Hkv, P, D, shift;           // P = 1 << shift
    const int32_t* table;           // [B, max_pages]
    int64_t table_stride;
    const int32_t* lens;            // [B]
    const int32_t* cu;              // [B + 1] or null (token b belongs to sequence b)
    int B, max_pages, max_new, max_kv;
    int64_t T;
    Dt dt;
};
// pages of one sequence that n new tokens can touch
inline int64_t pages_touched(int64_t n, int P) { return n <= 0 ? 0 : (n + P - 2) / P + 1; }
// The pages of all sequences that the call's tokens can lie in, in a row: as many
// places for each as max_new tokens can touch, or, where those are fewer, places by
// the call's tokens: sequence b's from first_place(cu[b], b) on. (n tokens touch at
// most (n + P - 2) / P + 1 pages, and first_place grows by n / P + 2 at least.) A
// prompt of 131072 tokens beside 255 single ones has 8703 places of 16 tokens so, by
// the former 2.1 million.
__host__ __device__ inline int64_t first_place(int cu, int b, int shift) { return (cu >> shift) + 2 * (int64_t)b; }
inline int64_t places_by_tokens(int64_t T, int B, int P) { return T / P + 2 * (int64_t)B; }
inline bool placed_by_tokens(const CacheArgs& c) {
    return c.cu && c.B * pages_touched(c.max_new, c.P) > places_by_tokens(c.T, c.B, c.P);
}
// workgroups of the append and of the read
inline int64_t cache_copy_blocks(const CacheArgs& c) {
    const int64_t places =
        placed_by_tokens(c) ? places_by_tokens(c.T, c.B, c.P) : c.B * pages_touched(c.max_new, c.P);
    return places * c.Hkv * 2;
}
hipError_t launch_cache_append(const CacheArgs& c, const Heads& k, const Heads& v, hipStream_t s);
hipError_t launch_cache_read(const CacheArgs& c, const Heads& k, const Heads& v, hipStream_t s);

// ---- attention over the cache -----------------------------------------------------
// Workgroups of k_attend_few that a compute unit holds. (Two tiles of rows of heads
// of 128 spill 24 bytes a lane so; 32 ragged sequences of 6 tokens of 4 heads took
// 74 us, at one workgroup without spills 112: loads in flight are what counts. For an
// fp32 q the pieces leave registers for one: the same in fp32 113.)
constexpr int few_held(int D, bool f32) { return D > 128 || f32 ? 1 : 2; }

// How one call is cut up: row tiles of `rows` (token, head) rows for each sequence
// and key head (few: one tile of 16 holds every sequence's). Shared: `blocks`
// workgroups take equal shares of all of them, and a row has up to `splits` parts.
// Otherwise: a workgroup for each tile and each of `splits` ranges of `chunk` keys
// (the last one open). With more than one split partial results go to the workspace
// and a second kernel joins them. (Shared: chunk is the least share's keys.)
struct AttnPlan {
    bool few, pair;                 // every sequence's rows fit a tile of 16, two of them
    bool shared;
    int waves;                      // of the row-tile kernel's workgroups (32 rows each)
    int pieces;                     // bf16 pieces of the weights of a bf16 q there, at least
    int rows, splits;
    int64_t row_tiles, chunk, blocks;
    size_t ws_bytes;                // 0 with one split
};

// Sequences of up to so many rows a key head keep the weights of a bf16 q to 16 bits,
// in every kernel.
constexpr int kPreciseRows = 128;

// Calls of up to so many rows are shared out evenly, whatever their lengths, and
// joined (a join of 32768 rows takes 15 us); larger ones have row tiles to fill the
// chip without, and shares of theirs are uneven (6 prompts of 30 to 1500 tokens, 28
// heads: 285 us shared, 217 as a workgroup for each row tile). Below, with the join,
// shared and as a workgroup for each range of keys: 32 ragged sequences of 60 tokens
// of 4 heads 207 and 506 us; 64 tokens beside 31 single ones 182 and 497, 512 beside
// them 437 and 928; 6 prompts of up to 150 tokens 55 and 64; 256 tokens over 32768
// keys 147 and 165; 32 tokens of one sequence, where every length is the same, 47 and
// 47.
constexpr int64_t kSharedRows = 32768;
// The parts of rows take up to so much workspace in any call. Few sequences stay far
// below it (32 of 32768 keys, 32 heads of 128: 34 MiB); many need few parts each,
// since the shares are then longer than a sequence.
constexpr int64_t kPartBytes = (int64_t)256 << 20;

inline AttnPlan attn_plan(const CacheArgs& c, int Hq, int window) {
    AttnPlan p{};
    const int64_t G = Hq / c.Hkv, most = (int64_t)c.max_new * G;
    p.few = most <= 16;
    // two tiles of 16 rows: 5 tokens of 4 heads over 32768 keys 24.6 us, by a row tile
    // of 128 33 (heads of 256 have no registers for it)
    p.pair = !p.few && most <= 32 && c.D <= 128;
    p.waves = c.D > 128 || c.dt == Dt::F32 || most <= 128 ? 4 : 8;
    p.pieces = most <= kPreciseRows ? 2 : 1;
    p.rows = p.few ? 16 : p.pair ? 32 : 32 * p.waves;
    p.row_tiles = (most + p.rows - 1) / p.rows;
    // keys that one row tile sees: all, or the window of its tokens
    int64_t span = c.max_kv > 0 ? c.max_kv : 1;
    if (window > 0) {
        const int64_t seen = (int64_t)window + p.rows / G + 1 + 63;
        if (seen < span) span = seen;
    }
    const int64_t whole = (int64_t)c.B * c.Hkv * p.row_tiles, rows = c.T * Hq;
    // parts of every row that kPartBytes hold
    const int64_t room = (kPartBytes / 4 / rows - 1) / (c.D + 2);
    const int64_t steps = (span + 63) / 64, all_steps = ((int64_t)c.max_pages * c.P + c.max_new) / 64 + 16;
    p.shared = p.few || p.pair || (rows <= kSharedRows && whole <= ((int64_t)1 << 31) / all_steps);
    if (p.shared) {
        // no share is less than 8 steps of 64 keys (see share_work); the chip holds one
        // workgroup a compute unit of the largest kinds, else two
        const int64_t held = p.few || p.pair ? few_held(c.D, c.dt == Dt::F32)
                                             : c.D > 128 || c.dt == Dt::F32 || p.waves == 8 ? 1 : 2;
        p.chunk = 8 * 64;
        p.splits = steps <= 8 ? 1 : (int)(steps / 8 + 2);
        if (p.splits > room) p.splits = room < 2 ? 1 : (int)room;
        const int64_t most_blocks = whole * ((steps + 7) / 8);
        p.blocks = (int64_t)compute_units() * held;
        if (most_blocks < p.blocks) p.blocks = most_blocks;
    } else {
        int64_t splits = whole > 0 ? (int64_t)compute_units() * 2 / whole : 1;
        const int64_t most_splits = (span + 511) / 512;
        if (splits > most_splits) splits = most_splits;
        if (splits > room) splits = room;
        if (splits < 1) splits = 1;
        p.chunk = ((span + splits - 1) / splits + 63) / 64 * 64;
        p.splits = (int)((span + p.chunk - 1) / p.chunk);
        p.blocks = whole * p.splits;
    }
    if (p.splits > 1) p.ws_bytes = (size_t)c.T * Hq * ((size_t)p.splits * (c.D + 2) + 1) * 4;
    return p;
}

hipError_t launch_cache_attention(const CacheArgs& c, const AttnPlan& plan, const Heads& q, int Hq, float scale,
                                  int window, const Heads& out, float* lse, void* ws, hipStream_t s);

}  // namespace sffn
