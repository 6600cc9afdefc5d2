// Softmax attention over packed sequences, forward.
//
//   S = scale q k^T (masked), O = softmax(S) v, L = log sum exp S   per head
// Row i of a causal sequence with nq queries and nk keys sees the keys
// j <= i + nk - nq. One pass over the keys with a running maximum m and sum l:
// for each tile of 64 keys, P = exp(S - m) and O <- O + P V; where a tile
// raises m by much, O and l are scaled down first. Rows that see nothing give
// O = 0 and L = -inf.
//
// Bound: the matrix unit, at the clock that the card's power allows. At 18432
// tokens, 24 heads of 128 (4.17 TFLOP): 3.49 ms, 1.20 PFLOP/s; the matrix
// unit is busy in 70 % of the cycles, at 1.65 GHz; LDS 35 %. 4608 tokens: 250 us,
// 1.04 PFLOP/s (432 tiles on 256 compute units). A tile costs 7 us of latency
// beside its steps: 1.2 to find its place, 3 for the loads, 1.2 for the first
// softmax, 1.3 for the stores.
// The same without the two wavefronts of a SIMD taking turns: 3.69 ms.
#include <hip/hip_runtime.h>

#include "attn_tile.h"

namespace ck4 {
namespace {

// A raised maximum is taken over only when it exceeds the held one by this
// much (in powers of two): until then P stays below 2^8, which fp32 sums and
// bf16 operands hold at full relative precision, and O is not rescaled.
constexpr float kSlack = 8.0f;
constexpr float kNoMax = -1e30f;

constexpr int kWaves = 8;
constexpr int kRows = kWaves * 32;  // of a tile
constexpr int kThreads = kWaves * 64;
// A partial result: the output sums, m and l of every lane.
template <int D>
constexpr int64_t kPartial = kThreads * (D / 2 + 2);

__device__ __forceinline__ float lse_of(float m, float l, float scale) {
    return l > 0.0f ? m * scale + logf(l) : l == 0.0f ? -INFINITY : l;
}

// The keys [64 from, 64 to) of one tile of queries.
template <int D>
__device__ __forceinline__ void attn_fwd_part(const Attn &a, const HeadsOut &out, float *lse, const Segment &g, int tile,
                                              float *partial, char *lds) {
    constexpr int WAVES = kWaves, kBytes = kTile * D * 2;
    const Span &s = g.s;
    const int head = g.head, kv = head / (a.hq / a.hk);
    const int thread = thread_again(), wave = __builtin_amdgcn_readfirstlane(thread / 64), lane = thread % 64, h = lane / 32;
    const int row0 = tile * kRows + wave * 32, row = row0 + lane % 32;
    // keys that the workgroup's, the wavefront's rows see at all, and all of them see
    const int last = tile * kRows + kRows - 1;
    const int end = limit(s, a.causal, last < s.nq ? last : s.nq - 1);
    const int wave_end = row0 < s.nq ? limit(s, a.causal, row0 + 31) : 0, wave_all = limit(s, a.causal, row0);
    const int mine = limit(s, a.causal, row);

    char *const own = lds + 4 * kBytes + wave * WaveRows<D>::kBytes;
    const WaveRows<D> q_rows(a.q.p + (s.q0 + row0) * a.q.st + head * a.q.sh, a.q.st, s.nq - row0, lane, a.d);
    u32x4 q_loaded[WaveRows<D>::kN];
    q_rows.load(q_loaded);

    const uint16_t *kp = a.k.p + s.k0 * a.k.st + kv * a.k.sh, *vp = a.v.p + s.k0 * a.v.st + kv * a.v.sh;
    const TileCopy<D, WAVES> kc(wave, lane, a.k.st, a.d), vc(wave, lane, a.v.st, a.d);
    const RowFrags<D> kf(lane);
    const ColFrags<D> vf(lane);
    // K of two tiles, then V of two tiles
    const auto issue_k = [&](int t) {
        kc.issue(kp + (int64_t)t * kTile * a.k.st, s.nk - t * kTile, a.k.st, a.d, lds + (t & 1) * kBytes);
    };
    const auto issue_v = [&](int t) {
        vc.issue(vp + (int64_t)t * kTile * a.v.st, s.nk - t * kTile, a.v.st, a.d, lds + (2 + (t & 1)) * kBytes);
    };

    f32x16 o[D / 32];
#pragma unroll
    for (int b = 0; b < D / 32; ++b)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[b][j] = 0.0f;
    float m = kNoMax, l = 0.0f;
    const float c = a.scale * kLog2e;

    bf16x8 q[D / 16];
    f32x16 p[2];
    // scores of tile t, unmasked, into zeros
    const auto scores = [&](int t, f32x16 x[2]) {
        const int kt = (t & 1) * kBytes;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 16; ++j) x[b][j] = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) x[b] = mfma(kf.get(lds, kt, b, i), q[i], x[b]);
        // fragments are read 6 products ahead
        __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);
#pragma unroll
        for (int i = 0; i < D / 8 - 6; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, 6, 0);
    };
    // the mask of tile t, and its maximum taken over into m if it is much above
    const auto raise = [&](int t, f32x16 x[2]) {
        if (t * kTile + kTile > wave_all) {
            const int left = mine - 1 - t * kTile - 4 * h;  // of the tile's keys, the last that the row sees
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int j = 0; j < 16; ++j) x[b][j] = masked(x[b][j], left - b * 32 - c_row(j, 0));
        }
        float top = x[0][0];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 16; ++j) top = fmaxf(top, x[b][j]);
        const float2 tops = both_halves(top);
        top = fmaxf(tops.x, tops.y);
        if (__any((top - m) * c > kSlack)) {
            const float up = fmaxf(m, top), f = __builtin_amdgcn_exp2f((m - up) * c);
            m = up;
            l *= f;
#pragma unroll
            for (int b = 0; b < D / 32; ++b)
#pragma unroll
                for (int j = 0; j < 16; ++j) o[b][j] *= f;
        }
    };
    // P goes to bf16, as V is: the matrix unit multiplies operands of one type, and fp32 at 1/16 of the rate. The sum l
    // takes the unrounded values. Against 64 bits the output is off by 0.0023 of itself, by 0.0017 if it alone were rounded.
    const auto weights = [&](const f32x16 x[2], bf16x8 w[4]) {
        const float mc = m * c;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x[r / 2][r % 2 * 8 + j], c, -mc));
                l += e;
                w[r][j] = (__bf16)e;
            }
    };
    const auto add = [&](int t, const bf16x8 w[4]) {
        const int vt = (2 + (t & 1)) * kBytes;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int b = 0; b < D / 32; ++b) o[b] = mfma(vf.get(lds, vt, b, r), w[r], o[b]);
        __builtin_amdgcn_sched_group_barrier(0x100, 8, 1);
#pragma unroll
        for (int i = 0; i < D / 8 - 4; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 1);
            __builtin_amdgcn_sched_group_barrier(0x100, 2, 1);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, 4, 1);
    };

    // Step t of a wavefront: the products S(t + 1) and O += P(t) V(t), a barrier, the softmax of S(t + 1), a barrier.
    // The two wavefronts of a SIMD (w and w + 4) take turns, one in its products (matrix unit), the other in its
    // softmax (vector unit): the later half of the wavefronts starts one barrier behind. Copies are issued at the start
    // of a softmax and waited for at its end, where nothing reads LDS; the buffers that they overwrite, K(t) and
    // V(t - 1), were read last half a step before.
    const int steps = (end + kTile - 1) / kTile, n = steps < g.to ? steps : g.to, from = g.from;
    const int wave_steps = (wave_end + kTile - 1) / kTile, nw = wave_steps < n ? wave_steps : n;
    const bool behind = wave >= WAVES / 2;
    bf16x8 w[4];
    const auto copy = [&](int t) {
        if (t + 2 < n) issue_k(t + 2);
        if (t + 1 < n) issue_v(t + 1);
    };
    const auto softmax = [&](int t) {
        raise(t, p);
        weights(p, w);
    };
    if (n > from) {
        issue_k(from);
        issue_v(from);
        if (n > from + 1) issue_k(from + 1);
        q_rows.fragments(q_loaded, own, kf, q);
        __syncthreads();
        if (nw > from) scores(from, p);
        __syncthreads();  // the first K is done with
        if (behind) copy(from);
        if (nw > from) softmax(from);
        if (behind) __syncthreads();
    }
    // The steps are peeled by what a wavefront still has to do: a condition around the products would cost copies of
    // their accumulators.
    int t = from;
    for (; t + 1 < nw; ++t) {
        __builtin_amdgcn_s_setprio(1);
        scores(t + 1, p);
        add(t, w);
        __builtin_amdgcn_s_setprio(0);
        __syncthreads();
        copy(behind ? t + 1 : t);
        softmax(t + 1);
        __syncthreads();
    }
    if (t < nw) {
        add(t, w);
        __syncthreads();
        copy(behind ? t + 1 : t);
        __syncthreads();
        ++t;
    }
    for (; t < n; ++t) {
        __syncthreads();
        copy(behind ? t + 1 : t);
        __syncthreads();
    }
    if (n > from && !behind) __syncthreads();
    const float2 ls = both_halves(l);
    l = ls.x + ls.y;
    if (partial) {
        store_partial<D / 32, kThreads>(o, partial);
        const auto ml = global(partial + kThreads * (D / 2) + thread);
        ml[0] = m;
        ml[kThreads] = l;
        return;
    }
    const WaveRows<D> o_rows(out.p + (s.q0 + row0) * out.st + head * out.sh, out.st, s.nq - row0, lane, a.d);
    o_rows.store(o, l > 0.0f ? 1.0f / l : l, own);
    if (lse && row < s.nq && h == 0) global(lse)[head * a.rows.tq + s.q0 + row] = lse_of(m, l, a.scale);
}

struct FwdArgs {
    Attn a;
    HeadsOut out;
    float *lse;
    Deal deal;
};

template <int D>
__global__ __launch_bounds__(kThreads, 2) void attn_fwd_kernel(FwdArgs) {
    __shared__ __align__(16) char lds[(4 * kTile + kRows) * D * 2];  // K of two tiles, V of two, Q and O
    Cursor cursor;
    while (!cursor.done) {
        const FwdArgs k = kernel_args<FwdArgs>();
        Segment g;
        float *partial;
        if (!next_segment<kRows, false, false>(blockIdx.x, gridDim.x, k.a.rows, k.a.causal, k.a.hq, 1, k.deal, kPartial<D>,
                                               cursor, &g, &partial))
            return;
        // causal: the last tiles have the most keys and go first
        const int tile = k.a.causal && !k.deal.partial ? g.s.tiles - 1 - g.s.tile : g.s.tile;
        attn_fwd_part<D>(k.a, k.out, k.lse, g, tile, partial, lds);
    }
}

// Joins the partial results of a tile, four of a lane's sums at a time; blockIdx.y: which of them.
template <int D>
__global__ __launch_bounds__(kThreads) void attn_fwd_join_kernel(Attn a, HeadsOut out, float *__restrict__ lse, Deal deal) {
    const int head = blockIdx.x / deal.tiles;
    Span s;
    if (!find_tile<kRows, false>(a.rows, blockIdx.x % deal.tiles, &s)) return;
    const Parts parts = Parts::of<kRows, false>(a.rows, a.causal, a.hq, 1, deal.most, s, head);
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64, h = lane / 32;
    const int row = s.tile * kRows + wave * 32 + lane % 32;
    if (!parts.cut() || row >= s.nq) return;
    const float c = a.scale * kLog2e;
    constexpr int kN = D / 8 / kJoinBlocks;
    f32x4 sum[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) sum[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float m = kNoMax, l = 0.0f;
#pragma unroll 4
    for (int w = parts.first; w <= parts.last; ++w) {
        const float *p = parts.at(deal.partial, w, kPartial<D>), *ml = p + kThreads * (D / 2) + threadIdx.x;
        const float up = fmaxf(m, ml[0]), f0 = __builtin_amdgcn_exp2f((m - up) * c),
                    f1 = __builtin_amdgcn_exp2f((ml[0] - up) * c);
        m = up;
        l = l * f0 + ml[kThreads] * f1;
#pragma unroll
        for (int i = 0; i < kN; ++i)
            sum[i] = sum[i] * f0 + reinterpret_cast<const f32x4 *>(p)[(blockIdx.y * kN + i) * kThreads + threadIdx.x] * f1;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int at = blockIdx.y * kN + i, e = at / 4 * 32 + c_row(at % 4 * 4, h);
        if (e < a.d)
            *reinterpret_cast<u32x2 *>(out.p + (int64_t)(s.q0 + row) * out.st + head * out.sh + e) =
                four(sum[i], l > 0.0f ? 1.0f / l : l);
    }
    if (lse && blockIdx.y == 0 && h == 0) lse[head * a.rows.tq + s.q0 + row] = lse_of(m, l, a.scale);
}

template <int D>
hipError_t launch_fwd(const Attn &a, const HeadsOut &out, float *lse, int most, float *partial, hipStream_t stream) {
    const int64_t tiles = most_tiles(a.rows.tq, kRows, a.rows.seqs, a.rows.cu_q != nullptr);
    const Deal deal{(int)tiles, most, partial};
    attn_fwd_kernel<D><<<dim3(grid_of(deal, a.hq)), kThreads, 0, stream>>>(FwdArgs{a, out, lse, deal});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !partial) return e;
    attn_fwd_join_kernel<D><<<dim3((unsigned)(tiles * a.hq), kJoinBlocks), kThreads, 0, stream>>>(a, out, lse, deal);
    return hipGetLastError();
}

}  // namespace

int64_t attention_floats(int seqs, int64_t tq, int64_t tk, int hq, int d) {
    return partial_floats(most_steps<kRows, false>(seqs, tq, tk, hq, 1), d <= 64 ? kPartial<64> : kPartial<128>);
}

hipError_t launch_attention(const Attn &a, const HeadsOut &out, float *lse, float *workspace, hipStream_t stream) {
    const int most = most_steps<kRows, false>(a.rows.seqs, a.rows.tq, a.rows.tk, a.hq, 1);
    float *partial = most ? workspace : nullptr;
    if (a.d <= 64) return launch_fwd<64>(a, out, lse, most, partial, stream);
    return launch_fwd<128>(a, out, lse, most, partial, stream);
}

}  // namespace ck4
