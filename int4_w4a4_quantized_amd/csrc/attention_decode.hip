// Attention of one new token per sequence over a key/value cache.
//
// HBM-bound: every filled slot of the cache is read once, 4 d bytes per key
// head, for 4 d operations per query head. 64 sequences of 300 to 16001 slots,
// 8 key heads of 128: 246 us, 5.4 TB/s; one sequence of 5003 slots: 11.1 us, and
// 4.0 us to join the parts, bound by launches and two rounds of copies' latency
// (4.9 tiles a piece on 4 wavefronts).
//
// The slots of all (sequence, key head) units form one line of 32-slot tiles, cut into equal pieces, one per
// workgroup, whatever the lengths: a piece may end inside a unit, and a unit
// may span many pieces. A workgroup that has all of a unit writes its output;
// otherwise it leaves a partial result (O, m, l), and a second kernel joins
// them in order. The query heads that share a key head are the columns of one
// product (16 at most; more are further units over the same slots).
#include <hip/hip_runtime.h>

#include "attn_tile.h"

namespace ck4 {
namespace {

constexpr int kSlots = 32;    // slots of a tile: one wavefront's
constexpr int kCols = 16;     // query heads of a unit
constexpr int kWaves = 4;     // of a workgroup on the line
constexpr int kGroups = 512;  // workgroups on the line at most
// Caches of up to kShort slots, by their size, as the lengths are on the device, are dealt whole units: no partial results
// and no second kernel, whose launch takes as long as the products. Up to kShorter with 4 wavefronts a unit, two workgroups a
// compute unit (64 sequences of 20 to 512 slots, 40/8 heads: 15.7 us, with 8 wavefronts 16.5), else with 8, which have 8 tiles
// each at most (full caches of 1024 slots: 16.7 us on the line, 11.8 with 8 and 11.9 with 4 wavefronts; 2048 slots: 16.6,
// 15.2, 20.3; 16 sequences of 100 to 2000: 23.3, 14.7, 17.5; 4096 slots: 16.0 on the line, 27.2 with 8 wavefronts).
constexpr int kShorter = 512, kShort = 2048;
constexpr float kSlackD = 8.0f;   // see attention.hip
constexpr float kNoMaxD = -1e30f;

__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Places of the 16-byte chunks of a row, as in attn_tile.h, for fragments of
// 16 rows: 8 rows x 32 bytes of a column read differ in their banks.
template <int D>
__device__ __forceinline__ int swz16(int r) {
    return D == 128 ? ((r & 7) << 1) | ((r >> 3) & 1) : (((r >> 1) & 3) << 1) | ((r >> 3) & 1);
}

__device__ __forceinline__ int filled(const Decode &a, int64_t b) {
    const int64_t n = a.lengths[b];
    return (int)(n < 0 ? 0 : n > a.slots ? a.slots : n);
}

// The line of tiles: sequence by sequence, in it unit by unit. It is cut into
// pieces of size or size + 1 tiles (the first `more` of them).
struct Line {
    int units;          // of a sequence: key heads x column blocks
    int total, pieces;  // fewer than 2^31 tiles: the entry point sees to it
    int size, more;

    __device__ __forceinline__ int start(int piece) const { return piece * size + (piece < more ? piece : more); }
    __device__ __forceinline__ int piece_of(int tile) const {
        const int big = more * (size + 1);
        return tile < big ? tile / (size + 1) : more + (tile - big) / size;
    }
};

__device__ __forceinline__ int tiles_of(const Decode &a, int64_t b) { return (filled(a, b) + kSlots - 1) / kSlots; }

__device__ __forceinline__ int wave_total(int v) {
#pragma unroll
    for (int step = 32; step > 0; step /= 2) v += __shfl_xor(v, step);
    return __builtin_amdgcn_readfirstlane(v);
}

// mine: the tiles of a unit of sequence `lane`.
__device__ __forceinline__ Line line_of(const Decode &a, int groups, int mine) {
    int n = mine;
    for (int64_t b = threadIdx.x % 64 + 64; b < a.batch; b += 64) n += tiles_of(a, b);
    Line l;
    l.units = a.hk * ((a.hq / a.hk + kCols - 1) / kCols);
    l.total = wave_total(n) * l.units;
    // Two workgroups a compute unit, as their LDS allows, or one where the pieces would be shorter than two rounds of
    // its wavefronts: half as many partial results (5003 slots, 8 key heads: 17.8 us, with two 20.6 us).
    const int some = groups / 2;
    l.pieces = l.total < some ? l.total : l.total < some * 2 * kWaves ? some : groups;
    if (l.pieces < 1) l.pieces = 1;
    l.size = l.total / l.pieces;
    l.more = l.total - l.size * l.pieces;
    return l;
}

// The sequence that tile `at` (< total) belongs to, and its first tile.
__device__ __forceinline__ int64_t find_sequence(const Decode &a, const Line &line, int mine, int at, int *start) {
    const int lane = threadIdx.x % 64;
    int before = 0;
    for (int64_t base = 0; base < a.batch; base += 64) {
        const int n = (base == 0 ? mine : base + lane < a.batch ? tiles_of(a, base + lane) : 0) * line.units;
        int upto = n;
#pragma unroll
        for (int step = 1; step < 64; step *= 2) {
            const int v = __shfl_up(upto, step);
            if (lane >= step) upto += v;
        }
        const uint64_t past = __ballot(before + upto > at);
        if (past) {
            const int l = __ffsll((unsigned long long)past) - 1;
            *start = before + __builtin_amdgcn_readlane(upto - n, l);
            return base + l;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    *start = before;
    return a.batch - 1;  // not reached for at < total
}

// All but the last n copies into LDS have arrived.
template <int N>
__device__ __forceinline__ void wait_copies() {
    static_assert(N < 16, "one field of the counter");
    __builtin_amdgcn_s_waitcnt(0x0F70 | N);
    asm volatile("" ::: "memory");
}
// All LDS reads have returned.
__device__ __forceinline__ void wait_reads() {
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
}

// Four column fragments: rows 4 g + 0..3 at each address, and 16 rows further.
// In one block with their wait: the compiler's own form of these reads waits
// for all copies into LDS too, also for those into other tiles.
template <int NEXT16>
__device__ __forceinline__ void read_columns(unsigned a0, unsigned a1, unsigned a2, unsigned a3, bf16x8 out[4]) {
    s16x4 r[8];
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8\n\tds_read_b64_tr_b16 %1, %8 offset:%12\n\t"
        "ds_read_b64_tr_b16 %2, %9\n\tds_read_b64_tr_b16 %3, %9 offset:%12\n\t"
        "ds_read_b64_tr_b16 %4, %10\n\tds_read_b64_tr_b16 %5, %10 offset:%12\n\t"
        "ds_read_b64_tr_b16 %6, %11\n\tds_read_b64_tr_b16 %7, %11 offset:%12\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(r[4]), "=&v"(r[5]), "=&v"(r[6]), "=&v"(r[7])
        : "v"(a0), "v"(a1), "v"(a2), "v"(a3), "n"(NEXT16)
        : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(r[2 * i], r[2 * i + 1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// A partial result: kCols rows of D sums, then m and l of every row. Piece w
// and unit u (over all sequences) meet at slot w + u: going along the line,
// one of the two grows by one at a time.
template <int D>
constexpr int kPartial = kCols * (D + 2);

// WHOLE: one workgroup a unit, no partial results.
template <int D, int WAVES, bool WHOLE>
__global__ __launch_bounds__(WAVES * 64, 2) void attn_decode_kernel(Decode a, float *__restrict__ partial, HeadsOut out,
                                                                     float *__restrict__ lse) {
    constexpr int kBytes = kSlots * D * 2;       // K or V tile
    constexpr int kLoads = kBytes / 1024;
    __shared__ __align__(16) char lds[WAVES][2 * kBytes];
    __shared__ float ms[WAVES][kCols], lsum[WAVES][kCols];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    const int col = lane % 16, g = lane / 16;
    const float c = a.scale * kLog2e;
    const int group = a.hq / a.hk, blocks = (group + kCols - 1) / kCols, piece = blockIdx.x;
    Line line{};
    int at = 0, end = 1, start = 0;
    int64_t b = 0;
    if constexpr (WHOLE) {
        b = piece / (a.hk * blocks);
    } else {
        const int first_tiles = lane < a.batch ? tiles_of(a, lane) : 0;
        line = line_of(a, (int)gridDim.x, first_tiles);
        if (line.total == 0 || piece >= line.pieces) return;
        at = line.start(piece);
        end = line.start(piece + 1);
        b = find_sequence(a, line, first_tiles, at, &start);
    }

    // a lane's source offsets and fragment places
    unsigned koff[kLoads], voff[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int pos = i * 1024 + lane * 16, row = pos / (2 * D), ch = pos % (2 * D) / 16 ^ swz16<D>(row % 16);
        koff[i] = 8 * ch < a.d ? (unsigned)(row * a.k.st * 2 + ch * 16) : 0x80000000u;
        voff[i] = 8 * ch < a.d ? (unsigned)(row * a.v.st * 2 + ch * 16) : 0x80000000u;
    }
    char *kt = lds[wave], *vt = kt + kBytes;
    const unsigned vt_at = (unsigned)(uintptr_t)(__attribute__((address_space(3))) char *)vt;
    int rat[D / 32], cat[D / 16];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) rat[i] = col * D * 2 + (((4 * i + g) ^ swz16<D>(col)) * 16);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const int row = 4 * g + col / 4, e = i * 16 + col % 4 * 4;
        cat[i] = row * D * 2 + ((e / 8 ^ swz16<D>(row)) * 16) + e % 8 * 2;
    }

    while (at < end) {
        int len = __builtin_amdgcn_readfirstlane(filled(a, b)), tiles = (len + kSlots - 1) / kSlots;
        while (!WHOLE && at - start >= tiles * line.units && b + 1 < a.batch) {  // on to the next sequence that has slots
            start += tiles * line.units;
            ++b;
            len = __builtin_amdgcn_readfirstlane(filled(a, b));
            tiles = (len + kSlots - 1) / kSlots;
        }
        const int unit = WHOLE ? piece % (a.hk * blocks) : (at - start) / tiles, kv = unit / blocks, block = unit % blocks;
        const int first = WHOLE ? 0 : at - start - unit * tiles;
        const int upto = !WHOLE && first + (end - at) < tiles ? first + (end - at) : tiles;
        const int heads = group - block * kCols < kCols ? group - block * kCols : kCols;
        const int head = kv * group + block * kCols + col;

        f32x4 o[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        float m = kNoMaxD, l = 0.0f;
        const uint16_t *kp = a.k.p + b * a.k_sb + kv * a.k.sh, *vp = a.v.p + b * a.v_sb + kv * a.v.sh;
        // K of the next tile is on its way during the softmax and the product with V, V during the next scores
        const auto copy = [&](const uint16_t *base, int64_t st, const unsigned *off, int t, char *to) {
            const int slot = t * kSlots, rows = len - slot < kSlots ? len - slot : kSlots;
            const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t *>(base + slot * st), (short)0,
                                                             (int)((rows - 1) * st * 2 + a.d * 2), 0x00020000);
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(
                    r, (__attribute__((address_space(3))) void *)(to + i * 1024), 16, (int)off[i], 0, 0, 0);
        };
        if (first + wave < upto) {
            copy(kp, a.k.st, koff, first + wave, kt);
            copy(vp, a.v.st, voff, first + wave, vt);
        }
        // after the first copies: their wait then covers q, and not the other way round
        bf16x8 q[D / 32];
        const uint16_t *qp = a.q.p + b * a.q.st + head * a.q.sh;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) q[i] = load_chunk(qp, 4 * i + g, a.d, col < heads);
        wait_copies<0>();  // here and not at the first use of q, which is in the loop
        for (int t = first + wave; t < upto; t += WAVES) {
            const bool more = t + WAVES < upto;
            const int slot = t * kSlots, rows = len - slot < kSlots ? len - slot : kSlots;
            wait_copies<kLoads>();  // K is there, V may be on its way: the wavefront's own tiles, no one else's
            f32x4 p[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                p[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < D / 32; ++i)
                    p[n] = mfma16(*reinterpret_cast<const bf16x8 *>(kt + rat[i] + n * 16 * D * 2), q[i], p[n]);
            }
            wait_reads();
            if (more) copy(kp, a.k.st, koff, t + WAVES, kt);
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (n * 16 + 4 * g + j >= rows) p[n][j] = -INFINITY;
                    top = fmaxf(top, p[n][j]);
                }
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            if (__any((top - m) * c > kSlackD)) {
                const float up = fmaxf(m, top), f = __builtin_amdgcn_exp2f((m - up) * c);
                m = up;
                l *= f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) o[i] *= f;
            }
            const float mc = m * c;
            bf16x8 w;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(p[n][j], c, -mc));
                    l += e;
                    w[4 * n + j] = (__bf16)e;  // for the product with V, as in attention.hip
                }
            if (more)
                wait_copies<kLoads>();  // V is there, the next K may be on its way
            else
                wait_copies<0>();
#pragma unroll
            for (int i = 0; i < D / 16; i += 4) {
                bf16x8 v[4];
                read_columns<16 * D * 2>(vt_at + cat[i], vt_at + cat[i + 1], vt_at + cat[i + 2], vt_at + cat[i + 3], v);
#pragma unroll
                for (int n = 0; n < 4; ++n) o[i + n] = mfma16(v[n], w, o[i + n]);
            }
            if (more) copy(vp, a.v.st, voff, t + WAVES, vt);
        }
        l += __shfl_xor(l, 16);
        l += __shfl_xor(l, 32);

        // join the wavefronts: each leaves O (row = head) in its own tiles' place
        constexpr int kRow = D + 4;  // padded: the 16 rows start in different banks
        float *mine = reinterpret_cast<float *>(lds[wave]);
        if (col < heads) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) *reinterpret_cast<f32x4 *>(mine + col * kRow + i * 16 + 4 * g) = o[i];
        }
        if (g == 0) {
            ms[wave][col] = m;
            lsum[wave][col] = l;
        }
        __syncthreads();
        const bool whole = WHOLE || (first == 0 && upto == tiles);
        float *part = partial + (piece + b * line.units + unit) * (int64_t)kPartial<D>;
        for (int i = threadIdx.x; i < heads * D; i += WAVES * 64) {
            const int r = i / D, e = i % D;
            float top = ms[0][r];
#pragma unroll
            for (int n = 1; n < WAVES; ++n) top = fmaxf(top, ms[n][r]);
            float sum = 0.0f, total = 0.0f;
#pragma unroll
            for (int n = 0; n < WAVES; ++n) {
                const float f = __builtin_amdgcn_exp2f((ms[n][r] - top) * c);
                sum = __builtin_fmaf(f, reinterpret_cast<const float *>(lds[n])[r * kRow + e], sum);
                total = __builtin_fmaf(f, lsum[n][r], total);
            }
            const int hd = kv * group + block * kCols + r;
            if (whole) {
                if (e < a.d) out.p[b * out.st + hd * out.sh + e] =
                    __builtin_bit_cast(uint16_t, (__bf16)(total > 0.0f ? sum / total : total));
                if (lse && e == 0)
                    lse[hd * a.batch + b] = total > 0.0f ? top * a.scale + logf(total) : total == 0.0f ? -INFINITY : total;
            } else {
                part[r * D + e] = sum;
                if (e == 0) {
                    part[kCols * D + r] = top;
                    part[kCols * D + kCols + r] = total;
                }
            }
        }
        if (WHOLE) return;
        __syncthreads();
        at += upto - first;
    }
}

// Joins the partial results of one sequence and query head: the pieces are
// dealt to the JOIN groups of D threads in turn, then the groups are added in order.
template <int D, int JOIN>
__global__ __launch_bounds__(D * JOIN) void attn_join_kernel(Decode a, int groups, const float *__restrict__ partial,
                                                              HeadsOut out, float *__restrict__ lse) {
    __shared__ float sums[JOIN][D], tops[JOIN], totals[JOIN];
    const int64_t b = blockIdx.x / a.hq;
    const int head = (int)(blockIdx.x % a.hq), e = threadIdx.x % D, g = threadIdx.x / D;
    const int group = a.hq / a.hk, blocks = (group + kCols - 1) / kCols;
    const int unit = head / group * blocks + head % group / kCols, r = head % group % kCols;
    const int tiles = tiles_of(a, b);
    float sum = 0.0f, total = 0.0f, top = kNoMaxD;
    const float c = a.scale * kLog2e;
    if (tiles > 0) {
        const int lane = threadIdx.x % 64, mine = lane < a.batch ? tiles_of(a, lane) : 0;
        const Line line = line_of(a, groups, mine);
        int before = lane < b ? mine : 0;
        for (int64_t i = lane + 64; i < b; i += 64) before += tiles_of(a, i);
        const int s = wave_total(before) * line.units + unit * tiles;
        const int w0 = line.piece_of(s), w1 = line.piece_of(s + tiles - 1);
        if (w0 == w1) return;  // written whole
        const float *p = partial + (b * line.units + unit) * (int64_t)kPartial<D>;
        constexpr int kAhead = JOIN > 1 ? 4 : 2;  // results read at once
        for (int w = w0 + g; w <= w1; w += kAhead * JOIN) {
            float o[kAhead], m[kAhead], l[kAhead], up = top;
#pragma unroll
            for (int n = 0; n < kAhead; ++n) {
                const int at = w + n * JOIN;
                const bool on = at <= w1;
                const float *x = p + (on ? at : w1) * (int64_t)kPartial<D>;
                const float xo = x[r * D + e], xm = x[kCols * D + r], xl = x[kCols * D + kCols + r];
                o[n] = on ? xo : 0.0f;
                m[n] = on ? xm : kNoMaxD;
                l[n] = on ? xl : 0.0f;
                up = fmaxf(up, m[n]);
            }
            const float f0 = __builtin_amdgcn_exp2f((top - up) * c);
            top = up;
            sum *= f0;
            total *= f0;
#pragma unroll
            for (int n = 0; n < kAhead; ++n) {
                const float f = __builtin_amdgcn_exp2f((m[n] - up) * c);
                sum = __builtin_fmaf(f, o[n], sum);
                total = __builtin_fmaf(f, l[n], total);
            }
        }
    }
    sums[g][e] = sum;
    if (e == 0) {
        tops[g] = top;
        totals[g] = total;
    }
    __syncthreads();
    if (g != 0) return;
#pragma unroll
    for (int n = 1; n < JOIN; ++n) top = fmaxf(top, tops[n]);
    sum = total = 0.0f;
#pragma unroll
    for (int n = 0; n < JOIN; ++n) {
        const float f = __builtin_amdgcn_exp2f((tops[n] - top) * c);
        sum = __builtin_fmaf(f, sums[n][e], sum);
        total = __builtin_fmaf(f, totals[n], total);
    }
    if (e < a.d) out.p[b * out.st + head * out.sh + e] =
        __builtin_bit_cast(uint16_t, (__bf16)(total > 0.0f ? sum / total : total));
    if (lse && e == 0)
        lse[head * a.batch + b] = total > 0.0f ? top * a.scale + logf(total) : total == 0.0f ? -INFINITY : total;
}

int64_t units_of(int hq, int hk) { return (int64_t)hk * ((hq / hk + kCols - 1) / kCols); }

template <int D>
hipError_t launch(const Decode &a, float *partial, const HeadsOut &out, float *lse, hipStream_t stream) {
    const int64_t units = a.batch * units_of(a.hq, a.hk);
    if (a.slots <= kShort) {
        if (a.slots <= kShorter)
            attn_decode_kernel<D, 4, true><<<dim3((unsigned)units), 4 * 64, 0, stream>>>(a, partial, out, lse);
        else
            attn_decode_kernel<D, 8, true><<<dim3((unsigned)units), 8 * 64, 0, stream>>>(a, partial, out, lse);
        return hipGetLastError();
    }
    attn_decode_kernel<D, kWaves, false><<<dim3(kGroups), kWaves * 64, 0, stream>>>(a, partial, out, lse);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // few units: each is spread over many pieces
    const dim3 grid((unsigned)(a.batch * a.hq));
    if (units * 4 <= kGroups)
        attn_join_kernel<D, 8><<<grid, D * 8, 0, stream>>>(a, kGroups, partial, out, lse);
    else
        attn_join_kernel<D, 1><<<grid, D, 0, stream>>>(a, kGroups, partial, out, lse);
    return hipGetLastError();
}

}  // namespace

int64_t attention_decode_floats(int64_t batch, int64_t slots, int hq, int hk, int d) {
    if (slots <= kShort) return 0;
    return (kGroups + batch * units_of(hq, hk)) * (d <= 64 ? kPartial<64> : kPartial<128>);
}

hipError_t launch_attention_decode(const Decode &a, float *partial, const HeadsOut &out, float *lse, hipStream_t stream) {
    if (a.d <= 64) return launch<64>(a, partial, out, lse, stream);
    return launch<128>(a, partial, out, lse, stream);
}

}  // namespace ck4
