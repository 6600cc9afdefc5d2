// How the attention kernels deal tiles to workgroups: the rows of a sequence,
// the steps that a tile takes, and the line of all steps that is cut into
// pieces where there are few tiles. Plain arithmetic, the same on the host,
// which sizes the workspace by it, and on the device.
#pragma once

#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "attn_kernels.h"

namespace ck4 {
namespace {

constexpr int kTile = 64;             // rows of a tile in LDS: a step

// One sequence's rows, and the tile of them that a workgroup has.
struct Span {
    int q0, k0;
    int nq, nk;
    int tile, tiles;
    int seq;
};

__host__ __device__ __forceinline__ int clamp_row(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// The rows from one start to the next, whatever the starts hold: inside the tensors. Sequences whose starts are out of
// order may claim the same rows.
__host__ __device__ __forceinline__ Span span_between(int tq, int tk, int q, int q_next, int k, int k_next) {
    Span s{};
    s.q0 = clamp_row(q, 0, tq);
    s.k0 = clamp_row(k, 0, tk);
    s.nq = clamp_row(q_next, s.q0, tq) - s.q0;
    s.nk = clamp_row(k_next, s.k0, tk) - s.k0;
    return s;
}

// Row `row` of a sequence sees the first limit() keys.
__host__ __device__ __forceinline__ int limit(const Span &s, bool causal, int row) {
    const int n = causal ? row - s.nq + s.nk + 1 : s.nk;
    return n < 0 ? 0 : n > s.nk ? s.nk : n;
}

// Upper bound of the tiles over all sequences with starts in order.
inline int64_t most_tiles(int64_t rows_total, int rows, int seqs, bool packed) {
    return (rows_total + rows - 1) / rows + (packed ? seqs : 0);
}

// Where there are too few tiles for the card's compute units, the steps of all
// tiles (64 keys each, or 64 queries of one head) form one line, which is cut
// into equal pieces, one per workgroup. A tile that no piece has whole is
// left as partial results and joined by a second kernel, in the order of the
// pieces. If no tile is much longer than a piece would be, whole tiles are
// dealt all the same.
//
// Steps of the tiles t of one sequence and head: c, or, in a causal sequence,
// clamp(a + B t, 1, c). A tile without any work counts as one step, so that its
// rows are written.
template <int B>
struct Ramp {
    int a, c;
    int tiles, mul;  // mul: the query heads of a key head, where they are walked one by one
    bool rising;

    __host__ __device__ __forceinline__ int steps(int t) const { return (rising ? clamp_row(a + B * t, 1, c) : c) * mul; }
    // steps of the tiles before t
    __host__ __device__ __forceinline__ int before(int t) const {
        // the first tiles with more than one step and with c, t at most
        const int n0 = rising ? clamp_row((B - a) / B, 0, t) : 0;
        const int n1 = rising ? clamp_row((c - a + B - 1) / B, n0, t) : 0;
        return (n0 + a * (n1 - n0) + B * ((n1 * (n1 - 1) - n0 * (n0 - 1)) / 2) + c * (t - n1)) * mul;
    }
};

// KEYS: tiles of ROWS keys, in falling order, stepping over queries; else
// tiles of ROWS queries stepping over keys.
template <int ROWS, bool KEYS>
__host__ __device__ __forceinline__ Ramp<ROWS / kTile> ramp_of(const Span &s, bool causal, int group) {
    static_assert(ROWS % kTile == 0, "whole steps");
    const int shift = s.nk - s.nq, walked = ((KEYS ? s.nq : s.nk) + kTile - 1) / kTile;
    Ramp<ROWS / kTile> r;
    r.tiles = ((KEYS ? s.nk : s.nq) + ROWS - 1) / ROWS;
    r.c = walked > 1 ? walked : 1;
    r.a = KEYS ? walked - (((r.tiles - 1) * ROWS - shift) >> 6) : (ROWS + shift + kTile - 1) >> 6;
    r.mul = KEYS ? group : 1;
    r.rising = causal;
    return r;
}

constexpr int kPieces = 256;  // one workgroup a compute unit: its 8 wavefronts of up to 256 registers fill it
constexpr int kLeast = 4;     // steps of a piece at least
// Tiles are cut where the longest takes at least so many steps more than a piece: the partial results and their
// joining take about as long.
constexpr int kGain = 16;
// From so many tiles on the compute units have work enough.
constexpr int64_t kFewTiles = 256;

// The steps of a launch's whole line at most, over all heads and sequences with starts in order; 0: whole tiles are dealt.
// Twice one more than it fits 32 bits.
template <int ROWS, bool KEYS>
inline int most_steps(int seqs, int64_t tq, int64_t tk, int heads, int group) {
    const int64_t tiles = most_tiles(KEYS ? tk : tq, ROWS, seqs, true) * heads;
    const int64_t steps = ((KEYS ? tq : tk) + kTile - 1) / kTile * group;
    return tiles >= kFewTiles || steps <= kGain || tiles * steps >= INT_MAX / 2 ? 0 : (int)(tiles * steps);
}

// The pieces that a line of `steps` steps is cut into at most.
__host__ __device__ __forceinline__ int most_pieces(int steps) {
    const int n = (steps + kLeast - 1) / kLeast;
    return n < kPieces ? n : kPieces;
}

// Floats of workspace of a launch with most_steps() `most`, of `each` floats a partial result.
inline int64_t partial_floats(int most, int64_t each) { return 2 * (int64_t)most_pieces(most) * each; }

// Two numbers of steps of at most most + 1, and their sum, in which all that is past `most` counts as most + 1.
__host__ __device__ __forceinline__ int add_steps(int a, int b, int most) { return a + b > most ? most + 1 : a + b; }

// What a line is cut by: its steps, and those of its longest tile.
struct LineSum {
    int total = 0, longest = 0;

    template <int B>
    __host__ __device__ __forceinline__ void add(const Ramp<B> &r, int heads, int most) {
        // one sequence alone never has more than `most`
        total = add_steps(total, r.before(r.tiles) * heads, most);
        if (r.tiles && r.steps(r.tiles - 1) > longest) longest = r.steps(r.tiles - 1);
    }
};

// The line cut into `count` pieces (0: whole tiles are dealt) of size or size + 1 steps, the first `more` of them.
// Sequences with starts out of order may claim rows more than once. A line that is longer than `most` by that is not
// cut, as the workspace would not hold its pieces' results.
struct Cut {
    int count, size, more;

    __host__ __device__ __forceinline__ Cut(const LineSum &s, int most) {
        count = most_pieces(s.total);
        size = s.total / (count > 1 ? count : 1);
        more = s.total - size * count;
        if (s.longest < size + kGain || s.total > most) count = 0;
    }
    __host__ __device__ __forceinline__ int start(int piece) const { return piece * size + (piece < more ? piece : more); }
    __host__ __device__ __forceinline__ int piece_of(int at) const {
        const int big = more * (size + 1);
        return at < big ? at / (size + 1) : more + (at - big) / size;
    }
    // The place of piece w's partial result: of the tile that it begins in, and of the one that it ends in.
    static __host__ __device__ __forceinline__ int place(int w, bool begins_in) { return 2 * w + (begins_in ? 0 : 1); }
};

// How a launch deals its tiles: each to a workgroup of its own (partial null), or, up to `most` steps in all, by pieces,
// whose partial results go to `partial`: piece w leaves at most two.
struct Deal {
    int tiles;  // upper bound, per head
    int most;
    float *partial;
};

// The workgroups of a launch: one a tile (over all heads), or one a piece.
inline unsigned grid_of(const Deal &d, int heads) {
    return (unsigned)(d.partial ? kPieces : ((int64_t)d.tiles * heads + 7) / 8 * 8);
}

}  // namespace
}  // namespace ck4
