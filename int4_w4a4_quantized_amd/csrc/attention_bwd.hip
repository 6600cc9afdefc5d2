// Gradients of softmax attention over packed sequences.
//
// With P = exp(scale q k^T - L) (masked) from the forward pass's L:
//   D_i = dO_i . O_i,  dV = P^T dO,  dS = P (dO V^T - D),
//   dQ = scale dS K,   dK = scale dS^T Q
// Two loops, each with one operand set held in registers and the other
// walked through LDS: one per tile of queries (dQ), one per tile of keys
// (dK, dV; the query heads that share a key head are summed in its registers).
// P is computed twice, 7 products instead of 5, and in exchange nothing is
// added through memory: no fp32 buffer for dQ, no atomics, and the results do
// not depend on the order in which workgroups run.
// P and dS are rounded to bf16 as operands of their products (the other
// operands are bf16 as well); all sums are fp32.
//
// Bound: the matrix unit's turns. At 4608 tokens, 24 heads of 128 (913 GFLOP in
// 7 products), calls apart, at about 2 GHz: 14 us for D, 634 us for the key tiles
// (820 TFLOP/s) and 389 us for the query tiles (1.01 PFLOP/s); 917 us for all
// three in a row of calls. Compute units work in 80 % of the time (432 tiles on
// 256 of them), the matrix unit in 48 % and 61 % of that.
#include <hip/hip_runtime.h>

#include "attn_tile.h"

namespace ck4 {
namespace {

constexpr int kWaves = 8;
constexpr int kRows = kWaves * 32;  // queries or keys of a tile
constexpr int kThreads = kWaves * 64;
// Partial results: dQ, or dK and dV.
template <int D>
constexpr int64_t kPartialQ = kThreads * (D / 2);
template <int D>
constexpr int64_t kPartialKV = kThreads * D;

// L log2(e) and D of every row: stat[head][row], stat[hq + head][row]. Rows that
// see nothing have L = -inf: +inf in its place makes every P of theirs zero.
// 16 lanes a row and head.
__global__ __launch_bounds__(256) void attn_stat_kernel(Heads o, Heads g, const float *__restrict__ lse, int64_t rows, int hq,
                                                        int d, float *__restrict__ stat) {
    const int64_t i = (int64_t)blockIdx.x * 16 + threadIdx.x / 16;
    const int c = threadIdx.x % 16;
    if (i >= rows * hq) return;
    const int64_t row = i / hq;
    const int head = (int)(i - row * hq);
    const bf16x8 of = load_chunk(o.p + row * o.st + head * o.sh, c, d, true);
    const bf16x8 gf = load_chunk(g.p + row * g.st + head * g.sh, c, d, true);
    float dot = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) dot = __builtin_fmaf((float)gf[e], (float)of[e], dot);
#pragma unroll
    for (int step = 1; step < 16; step *= 2) dot += __shfl_xor(dot, step);
    if (c == 0) {
        const float l = lse[head * rows + row] * kLog2e;
        stat[head * rows + row] = l == -INFINITY ? INFINITY : l;
        stat[(hq + head) * rows + row] = dot;
    }
}

// The keys [64 from, 64 to) for one tile of queries.
template <int D>
__device__ __forceinline__ void attn_dq_part(const Attn &a, const Heads &g, const float *stat, const HeadsOut &dq,
                                             const Segment &seg, int tile, float *partial, char *lds) {
    constexpr int WAVES = kWaves, kBytes = kTile * D * 2;
    const Span &s = seg.s;
    const int head = seg.head, kv = head / (a.hq / a.hk);
    const int thread = thread_again(), wave = __builtin_amdgcn_readfirstlane(thread / 64), lane = thread % 64, h = lane / 32;
    const int row0 = tile * kRows + wave * 32, row = row0 + lane % 32;
    const int last = tile * kRows + kRows - 1;
    const int end = limit(s, a.causal, last < s.nq ? last : s.nq - 1);
    const int wave_end = row0 < s.nq ? limit(s, a.causal, row0 + 31) : 0, wave_all = limit(s, a.causal, row0);
    const int mine = limit(s, a.causal, row);

    const bool on = row < s.nq;
    char *const own = lds + 5 * kBytes + wave * WaveRows<D>::kBytes;
    const WaveRows<D> q_rows(a.q.p + (s.q0 + row0) * a.q.st + head * a.q.sh, a.q.st, s.nq - row0, lane, a.d);
    const WaveRows<D> g_rows(g.p + (s.q0 + row0) * g.st + head * g.sh, g.st, s.nq - row0, lane, a.d);
    u32x4 q_loaded[WaveRows<D>::kN], g_loaded[WaveRows<D>::kN];
    q_rows.load(q_loaded);
    g_rows.load(g_loaded);
    bf16x8 qf[D / 16], gf[D / 16];
    const int64_t at = head * a.rows.tq + s.q0 + row;
    const float l2 = on ? global(stat)[at] : INFINITY, dot = on ? global(stat)[at + a.hq * a.rows.tq] : 0.0f;

    const uint16_t *kp = a.k.p + s.k0 * a.k.st + kv * a.k.sh, *vp = a.v.p + s.k0 * a.v.st + kv * a.v.sh;
    const TileCopy<D, WAVES> kc(wave, lane, a.k.st, a.d), vc(wave, lane, a.v.st, a.d);
    const RowFrags<D> rf(lane);
    const ColFrags<D> cf(lane);
    f32x16 acc[D / 32];
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[b][j] = 0.0f;
    const float c = a.scale * kLog2e;
    const int steps = (end + kTile - 1) / kTile, n = steps < seg.to ? steps : seg.to, from = seg.from;
    const int wave_steps = (wave_end + kTile - 1) / kTile, nw = wave_steps < n ? wave_steps : n;
    const bool behind = wave >= WAVES / 2;

    // K of three tiles, V of two
    const auto copy = [&](int t, int k_slot) {
        if (t < n) {
            kc.issue(kp + (int64_t)t * kTile * a.k.st, s.nk - t * kTile, a.k.st, a.d, lds + k_slot * kBytes);
            vc.issue(vp + (int64_t)t * kTile * a.v.st, s.nk - t * kTile, a.v.st, a.d, lds + (3 + (t & 1)) * kBytes);
        }
    };
    f32x16 p[2], dp[2];
    bf16x8 w[4];
    const auto scores = [&](int t, int k_slot) {
        const int kt = k_slot * kBytes, vt = (3 + (t & 1)) * kBytes;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 16; ++j) p[b][j] = dp[b][j] = 0.0f;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                p[b] = mfma(rf.get(lds, kt, b, i), qf[i], p[b]);
                dp[b] = mfma(rf.get(lds, vt, b, i), gf[i], dp[b]);
            }
        __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
        for (int i = 0; i < D / 4 - 6; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, 6, 0);
    };
    const auto add = [&](int k_slot) {
        const int kt = k_slot * kBytes;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int e = 0; e < D / 32; ++e) acc[e] = mfma(cf.get(lds, kt, e, r), w[r], acc[e]);
        __builtin_amdgcn_sched_group_barrier(0x100, 6, 1);
#pragma unroll
        for (int i = 0; i < D / 8 - 3; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 1);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 1);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, 3, 1);
    };
    const auto weights = [&](int t) {
        if (t * kTile + kTile > wave_all) {
            const int left = mine - 1 - t * kTile - 4 * h;  // of the tile's keys, the last that the row sees
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 16; ++j) p[b][j] = masked(p[b][j], left - b * 32 - c_row(j, 0));
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 16; ++j)
                p[b][j] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[b][j], c, -l2)) * (dp[b][j] - dot);
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = to_operand(p[r / 2], r % 2);
    };
    // The wavefronts of a SIMD take turns as in the forward kernel. K(t) is read twice, by the scores and a step later by
    // the sum of dQ, so there are three of them.
    int k0 = 0, k1 = 1, k2 = 2;  // places of K(t), K(t + 1), K(t + 2)
    if (n > from) {
        copy(from, 0);
        copy(from + 1, 1);
        q_rows.fragments(q_loaded, own, rf, qf);
        g_rows.fragments(g_loaded, own, rf, gf);
        __syncthreads();
        if (nw > from) scores(from, 0);
        __syncthreads();
        if (behind) copy(from + 2, 2);
        if (nw > from) weights(from);
        if (behind) __syncthreads();
    }
    const auto rest = [&](int t) {  // what follows the products of step t
        __syncthreads();
        if (behind)
            copy(t + 3, k0);
        else
            copy(t + 2, k2);
    };
    const auto turn = [&]() {
        const int k = k0;
        k0 = k1;
        k1 = k2;
        k2 = k;
        __syncthreads();
    };
    int t = from;
    for (; t + 1 < nw; ++t) {  // peeled as in the forward kernel
        __builtin_amdgcn_s_setprio(1);
        add(k0);
        scores(t + 1, k1);
        __builtin_amdgcn_s_setprio(0);
        rest(t);
        weights(t + 1);
        turn();
    }
    if (t < nw) {
        add(k0);
        rest(t);
        turn();
        ++t;
    }
    for (; t < n; ++t) {
        rest(t);
        turn();
    }
    if (n > from && !behind) __syncthreads();
    if (partial) {
        store_partial<D / 32, kThreads>(acc, partial);
        return;
    }
    const WaveRows<D> out(dq.p + (s.q0 + row0) * dq.st + head * dq.sh, dq.st, s.nq - row0, lane, a.d);
    out.store(acc, a.scale, own);
}

template <int D>
struct KeysLds {
    __align__(16) char rows[4 * kTile * D * 2];              // Q, dO of two tiles
    __align__(16) char v[kRows * D * 2];                     // V of the workgroup's keys
    __align__(16) float stat[2][2][kTile];                   // L log2(e), D of two tiles
};

// The steps [from, to) for one tile of keys: the tiles of 64 queries that see
// any of its keys, for each query head of the key head in turn.
template <int D>
__device__ __forceinline__ void attn_dkv_part(const Attn &a, const Heads &g, const float *stat, const HeadsOut &dk,
                                              const HeadsOut &dv, const Segment &seg, float *partial, KeysLds<D> &mem) {
    constexpr int WAVES = kWaves, kBytes = kTile * D * 2;
    const Span &s = seg.s;
    const int kv = seg.head;
    char *const lds = mem.rows, *const vl = mem.v;
    float (&rows)[2][2][kTile] = mem.stat;
    const int thread = thread_again(), wave = __builtin_amdgcn_readfirstlane(thread / 64), lane = thread % 64, h = lane / 32;
    const int key0 = s.tile * kRows + wave * 32, key = key0 + lane % 32;
    const int shift = s.nk - s.nq;
    const bool on = key < s.nk;
    const uint16_t *kp = a.k.p + (s.k0 + key) * a.k.st + kv * a.k.sh;
    bf16x8 kf[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) kf[i] = load_chunk(kp, 2 * i + h, a.d, on);
    {  // V of the workgroup's keys stays in LDS; tiles past the sequence are never read into anything that is stored
        const TileCopy<D, WAVES> vc(wave, lane, a.v.st, a.d);
        const uint16_t *vp = a.v.p + (s.k0 + s.tile * kRows) * a.v.st + kv * a.v.sh;
#pragma unroll
        for (int i = 0; i < kRows / kTile; ++i) {
            const int left = s.nk - s.tile * kRows - i * kTile;
            if (left > 0) vc.issue(vp + (int64_t)i * kTile * a.v.st, left, a.v.st, a.d, vl + i * kBytes);
        }
    }
    const TileCopy<D, WAVES> qc(wave, lane, a.q.st, a.d), gc(wave, lane, g.st, a.d);
    const RowFrags<D> rf(lane);
    const ColFrags<D> cf(lane);
    f32x16 ak[D / 32], av[D / 32];
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int j = 0; j < 16; ++j) ak[b][j] = av[b][j] = 0.0f;
    const float c = a.scale * kLog2e;

    // causal: query i sees key j where i >= j - shift
    const auto first_row = [&](int j) { return a.causal && j > shift ? j - shift : 0; };
    const int t0 = first_row(s.tile * kRows) / kTile, per_head = (s.nq + kTile - 1) / kTile - t0;
    const int wave_all = first_row(key0 + 31), mine = first_row(key);
    const int group = a.hq / a.hk, all = per_head > 0 ? per_head * group : 0;
    const int from = seg.from, n = all < seg.to ? all : seg.to;
    const bool behind = wave >= WAVES / 2;
    const auto copy = [&](int it) {
        if (it >= n) return;
        const int head = kv * group + it / per_head, t = t0 + it % per_head, left = s.nq - t * kTile;
        const int64_t r = s.q0 + (int64_t)t * kTile;
        char *at = lds + (it & 1) * 2 * kBytes;
        qc.issue(a.q.p + r * a.q.st + head * a.q.sh, left, a.q.st, a.d, at);
        gc.issue(g.p + r * g.st + head * g.sh, left, g.st, a.d, at + kBytes);
        // one wavefront of each half: the halves copy at different times. Rows past the end: zeros, like their Q and dO
        const int which = wave % (WAVES / 2);
        if (which == 0) {
            const float *p = stat + ((int64_t)behind * a.hq + head) * a.rows.tq + r;
            const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(p), (short)0,
                                                              (left < kTile ? left : kTile) * 4, 0x00020000);
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rs, (__attribute__((address_space(3))) void *)(rows[it & 1][behind]), 4, lane * 4, 0, 0, 0);
        }
    };
    // block u: the 32 rows u % 2 of tile u / 2
    const auto row_of = [&](int u) { return (t0 + u / 2 % per_head) * kTile + u % 2 * 32; };
    f32x16 p, ds;
    bf16x8 wp[2], ws[2];
    const int vt = wave / 2 * kBytes;
    const auto scores = [&](int u) {
        const int qt = (u / 2 & 1) * 2 * kBytes, gt = qt + kBytes;
#pragma unroll
        for (int j = 0; j < 16; ++j) p[j] = ds[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            p = mfma(rf.get(lds, qt, u % 2, i), kf[i], p);
            ds = mfma(rf.get(lds, gt, u % 2, i), rf.get(vl, vt, wave % 2, i), ds);
        }
        __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
        for (int i = 0; i < D / 8 - 4; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, 4, 0);
    };
    const auto add = [&](int u) {
        const int qt = (u / 2 & 1) * 2 * kBytes, gt = qt + kBytes;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < D / 32; ++e) {
                av[e] = mfma(cf.get(lds, gt, e, 2 * (u % 2) + r), wp[r], av[e]);
                ak[e] = mfma(cf.get(lds, qt, e, 2 * (u % 2) + r), ws[r], ak[e]);
            }
        __builtin_amdgcn_sched_group_barrier(0x100, 6, 1);
#pragma unroll
        for (int i = 0; i < D / 8 - 3; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 1);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 1);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, 3, 1);
    };
    const auto weights = [&](int u) {
        const int q0 = row_of(u);
        if (q0 < wave_all) {
            const int past = q0 + 4 * h - mine;  // rows past the first that sees the lane's key
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = masked(p[j], past + c_row(j, 0));
        }
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const f32x4 l2 = *reinterpret_cast<const f32x4 *>(&rows[u / 2 & 1][0][u % 2 * 32 + c_row(j, h)]);
            const f32x4 dd = *reinterpret_cast<const f32x4 *>(&rows[u / 2 & 1][1][u % 2 * 32 + c_row(j, h)]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                p[j + i] = __builtin_amdgcn_exp2f(__builtin_fmaf(p[j + i], c, -l2[i]));
                ds[j + i] = p[j + i] * (ds[j + i] - dd[i]);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            wp[r] = to_operand(p, r);
            ws[r] = to_operand(ds, r);
        }
    };
    // The wavefronts of a SIMD take turns as in the forward kernel, in steps of one block.
    if (n > from) {
        copy(from);
        __syncthreads();
        scores(2 * from);
        if (behind) copy(from + 1);
        weights(2 * from);
        if (behind) __syncthreads();
    } else {
        __syncthreads();  // V has arrived, whose place the results go through
    }
    int u = 2 * from;
    for (; u + 1 < 2 * n; ++u) {
        __builtin_amdgcn_s_setprio(1);
        add(u);
        scores(u + 1);
        __builtin_amdgcn_s_setprio(0);
        __syncthreads();
        const int next = u + (behind ? 1 : 0);
        if (next % 2 == 0) copy(next / 2 + 1);
        weights(u + 1);
        __syncthreads();
    }
    if (u < 2 * n) {
        add(u);
        __syncthreads();
        __syncthreads();
    }
    if (n > from && !behind) __syncthreads();
    if (partial) {
        store_partial<D / 32, kThreads>(ak, partial);
        store_partial<D / 32, kThreads>(av, partial + kThreads * (D / 2));
    } else {
        char *const own = vl + wave * WaveRows<D>::kBytes;  // the wavefront's rows of V
        const WaveRows<D> k_out(dk.p + (s.k0 + key0) * dk.st + kv * dk.sh, dk.st, s.nk - key0, lane, a.d);
        const WaveRows<D> v_out(dv.p + (s.k0 + key0) * dv.st + kv * dv.sh, dv.st, s.nk - key0, lane, a.d);
        k_out.store(ak, a.scale, own);
        v_out.store(av, 1.0f, own);
    }
    __syncthreads();  // V is done with
}

struct BwdArgs {
    Attn a;
    Heads g;
    const float *stat;
    HeadsOut dq, dk, dv;
    Deal keys, queries;
    unsigned key_groups;  // workgroups of the key tiles, a multiple of 8
};

// The tiles of keys, then those of queries, in one launch where tiles are cut:
// query tiles fill up the compute units that the last key tiles leave idle
// (packed, 40/8 heads: 372 us in two, 342 in one); and where all of them run at
// once (one sequence of 672, 4 heads: 79 us in two launches, 50 in one). Else in
// a launch each, as the two loops get better code alone (4608 tokens, 24
// heads: 996 us in one, 926 in two).
enum Which { kBoth, kKeys, kQueries };
template <int D, Which W>
__global__ __launch_bounds__(kThreads, 2) void attn_bwd_kernel(BwdArgs) {
    constexpr int kQueryBytes = (5 * kTile + kRows) * D * 2;  // K of three tiles, V of two, and Q, dO and dQ in turn
    constexpr int kKeyBytes = sizeof(KeysLds<D>);
    __shared__ __align__(16) char mem[W == kKeys || (W == kBoth && kKeyBytes > kQueryBytes) ? kKeyBytes : kQueryBytes];
    Cursor cursor;
    Segment g;
    float *partial;
    if (W == kKeys || (W == kBoth && blockIdx.x < kernel_args<BwdArgs>().key_groups)) {
        while (!cursor.done) {
            const BwdArgs k = kernel_args<BwdArgs>();
            if (!next_segment<kRows, true, false>(blockIdx.x, k.key_groups, k.a.rows, k.a.causal, k.a.hk, k.a.hq / k.a.hk,
                                                  k.keys, kPartialKV<D>, cursor, &g, &partial))
                return;
            attn_dkv_part<D>(k.a, k.g, k.stat, k.dk, k.dv, g, partial, *reinterpret_cast<KeysLds<D> *>(mem));
        }
        return;
    }
    if constexpr (W != kKeys) while (!cursor.done) {
        const BwdArgs k = kernel_args<BwdArgs>();
        if (!next_segment<kRows, false, true>(blockIdx.x - k.key_groups, gridDim.x - k.key_groups, k.a.rows, k.a.causal,
                                              k.a.hq, 1, k.queries, kPartialQ<D>, cursor, &g, &partial))
            return;
        // causal: the last tiles have the most keys and go first
        const int tile = k.a.causal && !k.queries.partial ? g.s.tiles - 1 - g.s.tile : g.s.tile;
        attn_dq_part<D>(k.a, k.g, k.stat, k.dq, g, tile, partial, mem);
    }
}

// Joins the partial results of a tile, dQ or dK and dV, four of a lane's sums at a time; blockIdx.y: which of them.
template <int D, bool KEYS>
__device__ __forceinline__ void join_grads(const Attn &a, const HeadsOut &o0, const HeadsOut &o1, const Deal &deal, int item) {
    constexpr int64_t kEach = KEYS ? kPartialKV<D> : kPartialQ<D>;
    const int head = item / deal.tiles;
    Span s;
    if (!find_tile<kRows, KEYS>(a.rows, item % deal.tiles, &s)) return;
    const Parts parts =
        Parts::of<kRows, KEYS>(a.rows, a.causal, KEYS ? a.hk : a.hq, KEYS ? a.hq / a.hk : 1, deal.most, s, head);
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, h = lane / 32;
    const int row = s.tile * kRows + wave * 32 + lane % 32;
    if (!parts.cut() || row >= (KEYS ? s.nk : s.nq)) return;
    constexpr int kN = (KEYS ? D / 4 : D / 8) / kJoinBlocks;
    f32x4 sum[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) sum[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int w = parts.first; w <= parts.last; ++w) {
        const f32x4 *p = reinterpret_cast<const f32x4 *>(parts.at(deal.partial, w, kEach));
#pragma unroll
        for (int i = 0; i < kN; ++i) sum[i] += p[(blockIdx.y * kN + i) * kThreads + threadIdx.x];
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int at = blockIdx.y * kN + i;
        const bool second = at >= D / 8;
        const int n = second ? at - D / 8 : at, e = n / 4 * 32 + c_row(n % 4 * 4, h);
        const HeadsOut &out = second ? o1 : o0;
        if (e < a.d)
            *reinterpret_cast<u32x2 *>(out.p + (int64_t)((KEYS ? s.k0 : s.q0) + row) * out.st + head * out.sh + e) =
                four(sum[i], second ? 1.0f : a.scale);
    }
}

// The tiles of keys, then those of queries, as far as they are cut.
template <int D>
__global__ __launch_bounds__(kThreads) void attn_grad_join_kernel(BwdArgs k) {
    const int keys = k.keys.partial ? k.keys.tiles * k.a.hk : 0, item = (int)blockIdx.x;
    if (item < keys)
        join_grads<D, true>(k.a, k.dk, k.dv, k.keys, item);
    else
        join_grads<D, false>(k.a, k.dq, k.dq, k.queries, item - keys);
}

// Steps of the line of all tiles of queries, and of keys.
int most_q(int seqs, int64_t tq, int64_t tk, int hq) { return most_steps<kRows, false>(seqs, tq, tk, hq, 1); }
int most_kv(int seqs, int64_t tq, int64_t tk, int hq, int hk) { return most_steps<kRows, true>(seqs, tq, tk, hk, hq / hk); }

template <int D>
hipError_t launch_bwd(const Attn &a, const Heads &dout, const float *stat, float *part_q, float *part_kv, const HeadsOut &dq,
                      const HeadsOut &dk, const HeadsOut &dv, hipStream_t stream) {
    const Packed &r = a.rows;
    const bool packed = r.cu_q != nullptr;
    const Deal qd{(int)most_tiles(r.tq, kRows, r.seqs, packed), most_q(r.seqs, r.tq, r.tk, a.hq), part_q};
    const Deal kd{(int)most_tiles(r.tk, kRows, r.seqs, packed), most_kv(r.seqs, r.tq, r.tk, a.hq, a.hk), part_kv};
    const unsigned keys = grid_of(kd, a.hk), queries = grid_of(qd, a.hq);
    BwdArgs args{a, dout, stat, dq, dk, dv, kd, qd, keys};
    if (part_q || part_kv || keys + queries <= kPieces) {
        attn_bwd_kernel<D, kBoth><<<dim3(keys + queries), kThreads, 0, stream>>>(args);
    } else {
        attn_bwd_kernel<D, kKeys><<<dim3(keys), kThreads, 0, stream>>>(args);
        args.key_groups = 0;
        attn_bwd_kernel<D, kQueries><<<dim3(queries), kThreads, 0, stream>>>(args);
    }
    const hipError_t e = hipGetLastError();
    const unsigned cut = (part_kv ? kd.tiles * a.hk : 0) + (part_q ? qd.tiles * a.hq : 0);
    if (e != hipSuccess || cut == 0) return e;
    attn_grad_join_kernel<D><<<dim3(cut, kJoinBlocks), kThreads, 0, stream>>>(args);
    return hipGetLastError();
}

int64_t floats_q(int seqs, int64_t tq, int64_t tk, int hq, int d) {
    return partial_floats(most_q(seqs, tq, tk, hq), d <= 64 ? kPartialQ<64> : kPartialQ<128>);
}
int64_t floats_kv(int seqs, int64_t tq, int64_t tk, int hq, int hk, int d) {
    return partial_floats(most_kv(seqs, tq, tk, hq, hk), d <= 64 ? kPartialKV<64> : kPartialKV<128>);
}
int64_t floats_stat(int64_t tq, int hq) { return (2 * tq * hq + 3) / 4 * 4; }

}  // namespace

int64_t attention_backward_floats(int seqs, int64_t tq, int64_t tk, int hq, int hk, int d) {
    return floats_stat(tq, hq) + floats_q(seqs, tq, tk, hq, d) + floats_kv(seqs, tq, tk, hq, hk, d);
}

hipError_t launch_attention_backward(const Attn &a, const Heads &out, const Heads &dout, const float *lse, float *workspace,
                                     const HeadsOut &dq, const HeadsOut &dk, const HeadsOut &dv, hipStream_t stream) {
    const Packed &r = a.rows;
    attn_stat_kernel<<<dim3((unsigned)((r.tq * a.hq + 15) / 16)), 256, 0, stream>>>(out, dout, lse, r.tq, a.hq, a.d, workspace);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t nq = floats_q(r.seqs, r.tq, r.tk, a.hq, a.d), nkv = floats_kv(r.seqs, r.tq, r.tk, a.hq, a.hk, a.d);
    float *partial = workspace + floats_stat(r.tq, a.hq);
    float *part_q = nq ? partial : nullptr, *part_kv = nkv ? partial + nq : nullptr;
    if (a.d <= 64) return launch_bwd<64>(a, dout, workspace, part_q, part_kv, dq, dk, dv, stream);
    return launch_bwd<128>(a, dout, workspace, part_q, part_kv, dq, dk, dv, stream);
}

}  // namespace ck4
