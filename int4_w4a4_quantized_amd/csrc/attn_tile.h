// Building blocks of the attention kernels: the tile in LDS and its copy, the
// operand fragments of the matrix instructions, the place of a workgroup in
// packed sequences.
//
// A tile is 64 rows (keys or queries) of one head, row-major in LDS, D bf16
// elements a row, in 16-byte chunks. The chunk c of row r lies at place
// c ^ swz(r). Two kinds of reads go to it, and swz spreads both over all 64
// banks:
//   - row fragments (ds_read_b128): 32 lanes read one chunk of 32 rows;
//   - column fragments (ds_read_b64_tr_b16): 16 lanes read a 4-row x 16-element
//     block and get it transposed, a column of 4 rows each.
//
// The products are transposed so that softmax rows lie in lanes. With
// v_mfma_f32_32x32x16_bf16, C[i][j] sits in lane j % 32 + 32 h, register
// 4 (i / 8) + i % 4, h = (i / 4) % 2. Scores are computed as S^T = K Q^T: a
// lane holds 16 keys of one query, and the row maximum and sum are in-lane but
// for one exchange between the two lane halves. The 8 values of registers
// 8 n .. 8 n + 7, rounded to bf16, are at once the B operand of the next
// product, whose contraction runs over those keys: that operand wants 8 keys
// of one column per lane, and which 8 does not matter as long as the A operand
// brings the same, which the column fragments do (keys 4 h + 0..3 and
// 8 + 4 h + 0..3 of each 16). No value changes lanes between the products.
#pragma once

#include <hip/hip_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "attn_line.h"

namespace ck4 {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
__device__ __forceinline__ int swz(int r) {
    static_assert(D == 64 || D == 128, "rows of 128 or 256 bytes");
    return D == 128 ? ((r & 3) << 2) | ((r >> 2) & 3) : (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

// A lane's part of the copy of a tile into LDS: 16 bytes per instruction, the
// wavefront's 1 KB back to back in LDS, so the swizzle is applied on the side
// of the source. Rows past the descriptor's end and chunks past the head's d
// elements are out of range and arrive as zeros.
template <int D, int WAVES>
struct TileCopy {
    static constexpr int kBytes = kTile * D * 2;
    static constexpr int kPerWave = kBytes / 1024 / WAVES;
    static_assert(kPerWave >= 1, "too many waves for a tile");
    unsigned off[kPerWave];
    int wave;

    __device__ TileCopy(int wave_, int lane, int64_t stride, int d) : wave(wave_) {
#pragma unroll
        for (int i = 0; i < kPerWave; ++i) {
            const int pos = (wave * kPerWave + i) * 1024 + lane * 16;
            const int row = pos / (2 * D), c = pos % (2 * D) / 16 ^ swz<D>(row);
            off[i] = 8 * c < d ? (unsigned)(row * stride * 2 + c * 16) : 0x80000000u;
        }
    }
    // rows: the rows that exist from p on (at least 1); lds: the tile
    __device__ __forceinline__ void issue(const uint16_t *p, int rows, int64_t stride, int d, char *lds) const {
        const int n = rows < kTile ? rows : kTile;
        const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(p), (short)0,
                                                         (int)((n - 1) * stride * 2 + d * 2), 0x00020000);
#pragma unroll
        for (int i = 0; i < kPerWave; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                r, (__attribute__((address_space(3))) void *)(lds + (wave * kPerWave + i) * 1024), 16, (int)off[i], 0, 0, 0);
    }
};

// Keeps v in a register: it is not computed again where it is used.
__device__ __forceinline__ void pin(int &v) { asm volatile("" : "+v"(v)); }

// A lane's fragments of a tile that lies `tile` bytes (a multiple of its size)
// into an array in LDS. The places of a row's chunks differ by exclusive-ors
// with constants and are formed from one register as they are needed: held in
// a register each they made the backward kernels spill, and the forward kernel 2 % slower.
template <int D>
struct RowFrags {  // operand rows: 32 rows x 16 elements, lane = row, 8 elements from 8 h on
    int at;
    __device__ explicit RowFrags(int lane) {
        const int r = lane % 32, h = lane / 32;
        at = r * D * 2 + (h ^ swz<D>(r)) * 16;
        pin(at);
    }
    __device__ __forceinline__ bf16x8 get(const char *lds, int tile, int block32, int s) const {
        return *reinterpret_cast<const bf16x8 *>(lds + ((at + tile) ^ (32 * s)) + block32 * 32 * D * 2);
    }
};
template <int D>
struct ColFrags {  // operand columns: 32 elements x 16 rows, lane = element, rows 4 h + 0..3 and 8 + 4 h + 0..3
    int at[2];
    __device__ explicit ColFrags(int lane) {
        const int i = lane % 16, half16 = lane / 16 % 2, h = lane / 32;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int row = 8 * n + 4 * h + i / 4, e = half16 * 16 + i % 4 * 4;
            at[n] = row * D * 2 + (e / 8 ^ swz<D>(row)) * 16 + e % 8 * 2;
            pin(at[n]);
        }
    }
    __device__ __forceinline__ bf16x8 get(const char *lds, int tile, int b, int rows16) const {
        const s16x4 lo = read(lds + ((at[0] + tile) ^ (64 * b)) + rows16 * 16 * D * 2);
        const s16x4 hi = read(lds + ((at[1] + tile) ^ (64 * b)) + rows16 * 16 * D * 2);
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    static __device__ __forceinline__ s16x4 read(const char *p) {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(p));
    }
};

__device__ __forceinline__ f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Registers 8 n .. 8 n + 7 rounded to bf16: the B operand described above.
__device__ __forceinline__ bf16x8 to_operand(const f32x16 &c, int n) {
    bf16x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = (__bf16)c[8 * n + i];
    return r;
}

// Row of register j of C in its 32-row block, for lane half h.
__device__ __forceinline__ constexpr int c_row(int j, int h) { return 8 * (j / 4) + 4 * h + j % 4; }

// -inf in place of v where n is negative: sign arithmetic, as 32 lane masks would not fit the scalar registers.
__device__ __forceinline__ float masked(float v, int n) {
    const unsigned m = (unsigned)(n >> 31);
    return __uint_as_float((m & 0xFF800000u) | (~m & __float_as_uint(v)));
}

// x of this lane and of the lane 32 further: {lower half's, upper half's}.
__device__ __forceinline__ float2 both_halves(float x) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return {__uint_as_float(r[0]), __uint_as_float(r[1])};
}

// A pointer that is known to be to global memory: those read from a kernel's arguments again are not.
template <class T>
__device__ __forceinline__ auto global(T *p) {
    return (__attribute__((address_space(1))) T *)p;
}

// A lane's 8 elements of row p in chunk c of a head of d elements (zeros past them, or if !on).
__device__ __forceinline__ bf16x8 load_chunk(const uint16_t *p, int c, int d, bool on) {
    u32x4 v = {0, 0, 0, 0};
    if (on && 8 * c < d) v = *global(reinterpret_cast<const u32x4 *>(p + 8 * c));
    return __builtin_bit_cast(bf16x8, v);
}

// Four elements times `mul`, rounded to bf16.
__device__ __forceinline__ u32x2 four(f32x4 v, float mul) {
    bf16x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (__bf16)(v[i] * mul);
    return __builtin_bit_cast(u32x2, o);
}

// A wavefront's 32 rows of a head in memory, which its instructions reach as
// whole rows, 1 KB each; what the lanes hold of them as fragments or sums goes
// through 32 rows of LDS of the wavefront's own (laid out like a tile). Taken
// straight from the lanes, an instruction reaches 32 rows, a few bytes of each:
// 8 wavefronts' Q took 2.6 us to load and O 2.2 us to store.
// Rows past the head's end (`rows` exist; none or less: nothing does) and
// chunks past its d elements are read as zeros and not written.
template <int D>
struct WaveRows {
    static constexpr int kBytes = 32 * D * 2, kN = kBytes / 1024;
    __amdgpu_buffer_rsrc_t rsrc;
    int64_t stride;
    int lane, d;

    __device__ __forceinline__ WaveRows(const uint16_t *p, int64_t stride_, int rows, int lane_, int d_)
        : stride(stride_), lane(lane_), d(d_) {
        const int n = rows < 32 ? rows : 32;
        rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(p), (short)0,
                                                 n > 0 ? (int)((n - 1) * stride * 2 + d * 2) : 0, 0x00020000);
    }
    __device__ __forceinline__ int row(int i) const { return (i * 1024 + lane * 16) / (2 * D); }
    __device__ __forceinline__ int chunk() const { return lane * 16 % (2 * D) / 16; }
    __device__ __forceinline__ int offset(int i) const {
        return 8 * chunk() < d ? (int)(row(i) * stride * 2 + chunk() * 16) : INT_MIN;
    }
    __device__ __forceinline__ char *place(char *lds, int i) const {
        return lds + row(i) * 2 * D + (chunk() ^ swz<D>(row(i))) * 16;
    }
    static __device__ __forceinline__ void settle() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

    __device__ __forceinline__ void load(u32x4 v[kN]) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc, offset(i), 0, 0);
    }
    // the loaded rows as row fragments
    __device__ __forceinline__ void fragments(const u32x4 v[kN], char *lds, const RowFrags<D> &rf, bf16x8 f[D / 16]) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) *reinterpret_cast<u32x4 *>(place(lds, i)) = v[i];
        settle();
#pragma unroll
        for (int i = 0; i < D / 16; ++i) f[i] = rf.get(lds, 0, 0, i);
        settle();
    }
    // The columns of an accumulator set C[D elements][32 rows], times `mul` (the lane's row's), rounded to bf16.
    __device__ __forceinline__ void store(const f32x16 acc[D / 32], float mul, char *lds) const {
        const int r = lane % 32, h = lane / 32;
#pragma unroll
        for (int b = 0; b < D / 32; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<u32x2 *>(lds + r * 2 * D + ((b * 4 + j) ^ swz<D>(r)) * 16 + h * 8) =
                    four(f32x4{acc[b][4 * j], acc[b][4 * j + 1], acc[b][4 * j + 2], acc[b][4 * j + 3]}, mul);
        settle();
        u32x4 v[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = *reinterpret_cast<const u32x4 *>(place(lds, i));
        settle();
#pragma unroll
        for (int i = 0; i < kN; ++i) __builtin_amdgcn_raw_buffer_store_b128(v[i], rsrc, offset(i), 0, 0);
    }
};

// The thread's number, known anew: what is computed from it for one part of a tile is not kept for the next.
__device__ __forceinline__ int thread_again() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t & 1023;
}

// Exchanges within the wavefront, from lane numbers found by thread_again().
// What finds a workgroup's place is run once or twice a workgroup, from a cold
// instruction cache, so it is kept short: loops stay loops, numbers 32 bits.
__device__ __forceinline__ int from_lane(int v, int lane) { return __builtin_amdgcn_ds_bpermute(lane * 4, v); }
__device__ __forceinline__ int wave_sum(int v, int lane) {
#pragma unroll 1
    for (int step = 32; step > 0; step /= 2) v += from_lane(v, lane ^ step);
    return __builtin_amdgcn_readfirstlane(v);
}
__device__ __forceinline__ int wave_max(int v, int lane) {
#pragma unroll 1
    for (int step = 32; step > 0; step /= 2) v = max(v, from_lane(v, lane ^ step));
    return __builtin_amdgcn_readfirstlane(v);
}
// The sum of the values of the lanes up to this one.
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll 1
    for (int step = 1; step < 64; step *= 2) {
        const int o = from_lane(v, lane - step);
        v += lane >= step ? o : 0;
    }
    return v;
}

__device__ __forceinline__ Span span_of(const Packed &p, int i) {
    Span s{};
    if (p.cu_q) {
        const auto cu_q = global(p.cu_q), cu_k = global(p.cu_k);
        s = span_between((int)p.tq, (int)p.tk, cu_q[i], cu_q[i + 1], cu_k[i], cu_k[i + 1]);
    } else {
        s.nq = (int)p.tq;
        s.nk = (int)p.tk;
    }
    s.seq = i;
    return s;
}

// The same values in every lane, kept in scalar registers.
__device__ __forceinline__ Span uniform(Span s) {
    const auto u = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    return Span{u(s.q0), u(s.k0), u(s.nq), u(s.nk), u(s.tile), u(s.tiles), u(s.seq)};
}

// The tile'th tile of ROWS query rows (or key rows) over all sequences in
// order; false if there are fewer. Every wavefront finds it for itself.
template <int ROWS, bool KEYS>
__device__ __forceinline__ bool find_tile(const Packed &p, int tile, Span *out) {
    const int lane = thread_again() % 64;
#pragma unroll 1
    for (int base = 0; base < p.seqs; base += 64) {
        Span s{};
        if (base + lane < p.seqs) s = span_of(p, base + lane);
        const int n = ((KEYS ? s.nk : s.nq) + ROWS - 1) / ROWS;
        const int upto = wave_scan(n, lane);
        const uint64_t past = __ballot(upto > tile);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, l); };
            *out = Span{of(s.q0), of(s.k0), of(s.nq), of(s.nk), 0, of(n), base + l};
            out->tile = tile - (__builtin_amdgcn_readlane(upto, l) - out->tiles);
            return true;
        }
        tile -= __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// Workgroups are dealt to the 8 XCDs in turn. Work item of a workgroup such
// that each XCD has a contiguous range of the items (whole heads, mostly),
// whose keys and values then stay in its own L2. grid: a multiple of 8.
__device__ __forceinline__ int xcd_item(unsigned group, unsigned grid) { return (int)(group % 8 * (grid / 8) + group / 8); }

// The line of all steps, cut into pieces.
template <int ROWS, bool KEYS>
struct Pieces : Cut {
    const Packed &p;
    bool causal;
    int heads, group;

    static __device__ __forceinline__ Ramp<ROWS / kTile> ramp(const Packed &p, bool causal, int group, int i) {
        return ramp_of<ROWS, KEYS>(span_of(p, i), causal, group);
    }
    __device__ __forceinline__ int all_steps(int i) const {
        const auto r = ramp(p, causal, group, i);
        return r.before(r.tiles) * heads;
    }
    static __device__ __forceinline__ LineSum sum(const Packed &p, bool causal, int heads, int group, int most) {
        const int lane = thread_again() % 64;
        LineSum s;
#pragma unroll 1
        for (int i = lane; i < p.seqs; i += 64) s.add(ramp(p, causal, group, i), heads, most);
#pragma unroll 1
        for (int step = 32; step > 0; step /= 2) s.total = add_steps(s.total, from_lane(s.total, lane ^ step), most);
        s.total = __builtin_amdgcn_readfirstlane(s.total);
        s.longest = wave_max(s.longest, lane);
        return s;
    }
    __device__ __forceinline__ Pieces(const Packed &p_, bool causal_, int heads_, int group_, int most)
        : Cut(sum(p_, causal_, heads_, group_, most), most), p(p_), causal(causal_), heads(heads_), group(group_) {}
};

// A kernel's arguments (one struct), read again from where they are. Kernels that walk over several parts of tiles read
// them for each: kept across a part's steps, they would push the steps' own values out of the scalar registers.
template <class T>
__device__ __forceinline__ T kernel_args() {
    static_assert(sizeof(T) % 4 == 0, "whole words");
    struct Words {
        unsigned w[sizeof(T) / 4];
    } v;
    auto *p = (const __attribute__((address_space(4))) unsigned *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
#pragma unroll
    for (unsigned i = 0; i < sizeof(T) / 4; ++i) v.w[i] = p[i];
    return __builtin_bit_cast(T, v);
}

// A workgroup's part of a tile: steps [from, to).
struct Segment {
    Span s;
    int head;
    int from, to;
};

// A workgroup's way through its piece of the line: what is left of it, and the tile that it is in.
struct Cursor {
    int left = 0;
    int seq = 0, head = 0, t = 0;
    bool begins = true, done = false;
};

// ACROSS: the longest tiles of all heads of a causal call go before the shorter ones, instead of head by head (packed
// prompts, 40/8 heads: the kernel of dQ 5 % faster, the forward kernel 2 % slower).
// The next part of a tile that workgroup `group_id` of `groups` (a multiple of 8) has, and the place of its partial result
// (null: it is the whole tile); false if there is none.
template <int ROWS, bool KEYS, bool ACROSS>
__device__ __forceinline__ bool next_segment(unsigned group_id, unsigned groups, const Packed &p, bool causal, int heads,
                                             int group, const Deal &d, int64_t each, Cursor &c, Segment *g,
                                             float **partial) {
    int item = xcd_item(group_id, groups);
    bool whole = !d.partial;
    g->from = 0;
    g->to = INT_MAX;
    *partial = nullptr;
    if (!whole && c.begins) {
        const Pieces<ROWS, KEYS> pieces(p, causal, heads, group, d.most);
        whole = pieces.count == 0;
        if (!whole) {
            if (item >= pieces.count) return false;
            int at = pieces.start(item);
            c.left = pieces.start(item + 1) - at;
            const int lane = thread_again() % 64;
#pragma unroll 1
            for (int base = 0; base < p.seqs; base += 64) {
                const int n = base + lane < p.seqs ? pieces.all_steps(base + lane) : 0, upto = wave_scan(n, lane);
                const uint64_t past = __ballot(upto > at);
                if (past) {
                    const int l = __ffsll((unsigned long long)past) - 1;
                    c.seq = __builtin_amdgcn_readfirstlane(base + l);
                    at -= __builtin_amdgcn_readlane(upto - n, l);
                    break;
                }
                at -= __builtin_amdgcn_readlane(upto, 63);
            }
            const auto r = ramp_of<ROWS, KEYS>(uniform(span_of(p, c.seq)), causal, group);
            const int per_head = r.before(r.tiles);
            c.head = at / per_head;
            at -= c.head * per_head;
            int hi = r.tiles - 1;  // the last tile that starts at or before `at`
#pragma unroll 1
            while (c.t < hi) {
                const int mid = (c.t + hi + 1) / 2;
                if (r.before(mid) <= at)
                    c.t = mid;
                else
                    hi = mid - 1;
            }
            g->from = at - r.before(c.t);
        }
    }
    if (whole) {
        c.done = true;
        g->head = item / d.tiles;
        item %= d.tiles;
        if (ACROSS && causal && heads % 8 == 0) {  // all of an XCD's heads, tile by tile
            const int per_xcd = heads / 8, i = (int)group_id / 8;
            g->head = (int)group_id % 8 * per_xcd + i % per_xcd;
            item = i / per_xcd;
        }
        return g->head < heads && item < d.tiles && find_tile<ROWS, KEYS>(p, item, &g->s);
    }
    g->s = uniform(span_of(p, c.seq));
    auto r = ramp_of<ROWS, KEYS>(g->s, causal, group);
    if (!c.begins && ++c.t >= r.tiles) {  // on to the next head, or to the next sequence that has tiles
        c.t = 0;
        if (++c.head >= heads) {
            c.head = 0;
            do {
                if (++c.seq >= p.seqs) return false;
                g->s = uniform(span_of(p, c.seq));
                r = ramp_of<ROWS, KEYS>(g->s, causal, group);
            } while (r.tiles == 0);
        }
    }
    const int steps = r.steps(c.t);
    g->head = c.head;
    g->s.tile = KEYS ? r.tiles - 1 - c.t : c.t;
    g->s.tiles = r.tiles;
    g->to = min(g->from + c.left, steps);
    if (g->from > 0 || g->to < steps) *partial = d.partial + Cut::place(item, c.begins) * each;
    c.left -= g->to - g->from;
    c.begins = false;
    c.done = c.left <= 0;
    return true;
}

// The partial results of a tile, in order.
struct Parts {
    int first, last;  // pieces; last <= first: none, the tile was written whole
    bool begins;      // the first piece begins with the tile

    template <int ROWS, bool KEYS>
    static __device__ __forceinline__ Parts of(const Packed &p, bool causal, int heads, int group, int most, const Span &s,
                                               int head) {
        Parts r{0, 0, false};
        const Pieces<ROWS, KEYS> pieces(p, causal, heads, group, most);
        if (pieces.count == 0) return r;
        const int lane = thread_again() % 64;
        int n = 0;
#pragma unroll 1
        for (int i = lane; i < s.seq; i += 64) n += pieces.all_steps(i);
        const auto ramp = ramp_of<ROWS, KEYS>(s, causal, group);
        const int t = KEYS ? ramp.tiles - 1 - s.tile : s.tile;
        const int at = wave_sum(n, lane) + head * ramp.before(ramp.tiles) + ramp.before(t);
        r.first = pieces.piece_of(at);
        r.last = pieces.piece_of(at + ramp.steps(t) - 1);
        r.begins = pieces.start(r.first) == at;
        return r;
    }
    __device__ __forceinline__ bool cut() const { return last > first; }
    __device__ __forceinline__ const float *at(const float *partial, int w, int64_t each) const {
        return partial + Cut::place(w, w != first || begins) * each;
    }
};
constexpr int kJoinBlocks = 8;  // workgroups a tile that share its partial results' values

// A set of N accumulators of a workgroup of THREADS as partial results, coalesced.
template <int N, int THREADS>
__device__ __forceinline__ void store_partial(const f32x16 acc[N], float *to) {
    const int thread = thread_again();
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            global(reinterpret_cast<f32x4 *>(to))[(b * 4 + j) * THREADS + thread] =
                f32x4{acc[b][4 * j], acc[b][4 * j + 1], acc[b][4 * j + 2], acc[b][4 * j + 3]};
}

}  // namespace
}  // namespace ck4
