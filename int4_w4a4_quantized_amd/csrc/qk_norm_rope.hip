// RMS norm of every query and key head with the rotary position rotation in
// the same pass, and its gradients.
//
//   r = 1 / sqrt(mean(x^2) + eps)       per head, over its d elements
//   y = x r w                           w: the norm weight of the head group
//   out pair j = y pair j turned by the angle position(axis(j)) freqs[j]
// Backward, from g = d out:
//   z = g turned back, u = z w, n = x r
//   dx = r (u - n mean(u n)),  dw = sum over tokens and heads of z n
//
// Both directions are one pass over the heads and HBM-bound: 4 bytes an
// element forward, 6 backward. 4608 tokens of 24 + 24 heads of 128: forward
// 21.7 us (5.2 TB/s), backward 35.1 us (4.8 TB/s) and 4.1 us for the join of
// the weight gradients. A head lives in GL lanes of one wavefront, 8
// elements (16 bytes) a lane, so its sums are a few cross-lane adds and no
// data is staged. All sums are fp32, and outputs are rounded to bf16 once.
//
// The angles are computed, not looked up: one sine and cosine per token and
// pair serve all heads of the token. position * freq is formed and reduced
// modulo one turn in fp64 (pairs/token is 1/100 of the work and fp32 would
// lose 2^-24 of the whole angle, 1e-3 rad at 2^14 turns), the sine of the
// remainder in fp32.
#include <hip/hip_runtime.h>

#include "attn_kernels.h"

namespace ck4 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHead = 256;
constexpr int kBlocks = 2048, kBlocksBwd = 1024;  // at most: 8 and 4 blocks of 4 wavefronts a compute unit
// Half-split rotations exchange elements between lanes through LDS: one fp32 row per head in flight.
constexpr int kExchange = 64 * 8;

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// How the pairs of a head lie in the 8-element chunks of its lanes.
enum Layout { kInterleaved = 0, kHalves = 1, kHalvesOdd = 2 };  // kHalves: pairs a multiple of 8

__device__ __forceinline__ void unpack8(const u32x4 v, float x[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ u32x4 pack8(const float x[8]) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bf16x2 p = {(__bf16)x[2 * i], (__bf16)x[2 * i + 1]};
        v[i] = __builtin_bit_cast(unsigned, p);
    }
    return v;
}

template <int MASK>
__device__ __forceinline__ float add_xor(float x) {
    return x + __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(x), 0x1F | (MASK << 10)));
}

// Sum over the GL lanes of a head, the same bits in each of them.
template <int GL>
__device__ __forceinline__ float head_sum(float x) {
    x = add_xor<1>(x);
    x = add_xor<2>(x);
    if constexpr (GL > 4) x = add_xor<4>(x);
    if constexpr (GL > 8) x = add_xor<8>(x);
    if constexpr (GL > 16) x = add_xor<16>(x);
    return x;
}

__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// What a wavefront does in one step: 64 / GL heads of one token, all of q's and
// then k's. The steps of all tokens form one line, cut into equal pieces, one
// per wavefront, whatever the numbers of tokens and heads.
struct Steps {
    int64_t begin, end;
    int64_t token;
    int head;  // first head of the step, 0 <= head < hq + hk
};

template <int GL>
__device__ __forceinline__ Steps steps_of(const NormRope &a) {
    const int per_token = (a.heads[0] + a.heads[1] + 64 / GL - 1) / (64 / GL);
    const int64_t total = a.tokens * per_token, waves = (int64_t)gridDim.x * (kThreads / 64);
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    Steps s;
    s.begin = w * total / waves;
    s.end = (w + 1) * total / waves;
    s.token = s.begin / per_token;
    s.head = (int)(s.begin - s.token * per_token) * (64 / GL);
    return s;
}

template <int GL>
__device__ __forceinline__ void next_step(const NormRope &a, int64_t &token, int &head) {
    head += 64 / GL;
    if (head >= a.heads[0] + a.heads[1]) {
        head = 0;
        ++token;
    }
}

// The rotation of a lane's 8 elements at one token: y[i] c[i] + (its partner) s[i],
// with the identity past the rotated pairs. Interleaved pairs need c, s of 4 pairs.
template <int L>
struct Turn {
    static constexpr int kN = L == kInterleaved ? 4 : 8;
    float c[kN], s[kN];

    // cs: LDS of the wavefront, half a head long. sign -1 turns back.
    __device__ __forceinline__ void set(const Rope &r, int64_t token, int half, int lane, bool live, float sign, float2 *cs) {
        const int64_t at = token * r.axes;
        for (int j = threadIdx.x % 64; j < half; j += 64) {
            float2 v = {1.0f, 0.0f};
            if (j < r.pairs) {
                int axis = 0;
#pragma unroll
                for (int a = 0; a < kMaxAxes - 1; ++a) axis += (a < r.axes - 1 && j >= r.end[a]) ? 1 : 0;
                const double pos = r.pos_f32 ? (double)static_cast<const float *>(r.pos)[at + axis]
                                             : (double)static_cast<const int32_t *>(r.pos)[at + axis];
                const double turns = pos * (double)r.freqs[j] * 0.15915494309189533577;
                sincospif((float)(2.0 * (turns - rint(turns))), &v.y, &v.x);
            }
            cs[j] = v;
        }
        wave_lds_order();
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int e = 8 * lane + i;
            int j = L == kInterleaved ? 4 * lane + i : e < r.pairs ? e : e - r.pairs;
            const bool on = live && (L == kInterleaved || e < 2 * r.pairs);
            const float2 v = on ? cs[j] : float2{1.0f, 0.0f};
            c[i] = v.x;
            s[i] = (L != kInterleaved && e < r.pairs ? -sign : sign) * v.y;
        }
        wave_lds_order();
    }

    // ex: the head's exchange row in LDS. Lanes past the head (not live) hold zeros and take part with slots of their own.
    __device__ __forceinline__ void apply(float y[8], int lane, int pairs, float *ex) const {
        if constexpr (L == kInterleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = y[2 * i], b = y[2 * i + 1];
                y[2 * i] = a * c[i] - b * s[i];
                y[2 * i + 1] = b * c[i] + a * s[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) ex[8 * lane + i] = y[i];
            wave_lds_order();
            float other[8];
            if constexpr (L == kHalves) {  // a chunk lies whole in the first half, the second or the rest
                const int e0 = 8 * lane, from = e0 < pairs ? e0 + pairs : e0 < 2 * pairs ? e0 - pairs : e0;
#pragma unroll
                for (int i = 0; i < 8; ++i) other[i] = ex[from + i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int e = 8 * lane + i;
                    other[i] = ex[e < pairs ? e + pairs : e < 2 * pairs ? e - pairs : e];
                }
            }
            wave_lds_order();
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] * c[i] + other[i] * s[i];
        }
    }
};

// A lane's weights: 8 of each head group, ones where there are none.
__device__ __forceinline__ void load_weights(const float *w, int lane, bool live, float out[8]) {
    typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
    f32x4u lo = {1.0f, 1.0f, 1.0f, 1.0f}, hi = lo;
    if (w && live) {
        lo = *reinterpret_cast<const f32x4u *>(w + 8 * lane);
        hi = *reinterpret_cast<const f32x4u *>(w + 8 * lane + 4);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        out[i] = lo[i];
        out[4 + i] = hi[i];
    }
}

template <int GL, int L>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(NormRope a, HeadsOut o0, HeadsOut o1) {
    __shared__ float2 cs[kThreads / 64][kMaxHead / 2];
    __shared__ float ex[L == kInterleaved ? 1 : kThreads / 64][L == kInterleaved ? 1 : kExchange];
    const int half = a.d / 2, heads = a.heads[0] + a.heads[1];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % GL, grp = threadIdx.x % 64 / GL;
    const bool live = 8 * lane < a.d;
    const float inv_d = 1.0f / (float)a.d;
    float *exr = &ex[L == kInterleaved ? 0 : wave][L == kInterleaved ? 0 : grp * GL * 8];
    Steps st = steps_of<GL>(a);
    if (st.begin >= st.end) return;

    const auto load = [&](int64_t token, int head) {
        u32x4 v = {0, 0, 0, 0};
        const int h = head + grp;
        if (h < heads && live) {
            const bool k = h >= a.heads[0];
            const uint16_t *p = (k ? a.x[1].p + token * a.x[1].st : a.x[0].p + token * a.x[0].st) +
                                (k ? (h - a.heads[0]) * a.x[1].sh : h * a.x[0].sh);
            v = *reinterpret_cast<const u32x4 *>(p + 8 * lane);
        }
        return v;
    };
    int64_t token = st.token;
    int head = st.head;
    u32x4 next = load(token, head);
    float w0[8], w1[8];
    load_weights(a.w[0], lane, live, w0);
    load_weights(a.w[1], lane, live, w1);
    Turn<L> turn;
    turn.set(a.rope, token, half, lane, live, 1.0f, cs[wave]);
    for (int64_t i = st.begin; i < st.end; ++i) {
        const u32x4 cur = next;
        int64_t token2 = token;
        int head2 = head;
        next_step<GL>(a, token2, head2);
        if (i + 1 < st.end) next = load(token2, head2);
        const int h = head + grp;
        const bool k = h >= a.heads[0];
        float x[8];
        unpack8(cur, x);
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(x[e], x[e], sum);
        const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(head_sum<GL>(sum), inv_d, a.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * r * (k ? w1[e] : w0[e]);
        turn.apply(x, lane, a.rope.pairs, exr);
        if (h < heads && live) {
            uint16_t *p = (k ? o1.p + token * o1.st : o0.p + token * o0.st) +
                          (k ? (h - a.heads[0]) * o1.sh : h * o0.sh);
            *reinterpret_cast<u32x4 *>(p + 8 * lane) = pack8(x);
        }
        if (token2 != token && i + 1 < st.end) turn.set(a.rope, token2, half, lane, live, 1.0f, cs[wave]);
        token = token2;
        head = head2;
    }
}

// Every lane keeps its sums of the weight gradients in registers: the lanes at
// one place of a head own the same 8 columns. A block's sums go to `partial`,
// and norm_dw_kernel adds the blocks in order, so the result does not depend
// on timing.
template <int GL, int L>
__global__ __launch_bounds__(kThreads) void norm_rope_bwd_kernel(NormRope a, Heads g0, Heads g1, HeadsOut o0, HeadsOut o1,
                                                                 float *__restrict__ partial) {
    constexpr int kRows = kThreads / GL;
    __shared__ float2 cs[kThreads / 64][kMaxHead / 2];
    __shared__ float ex[L == kInterleaved ? 1 : kThreads / 64][L == kInterleaved ? 1 : kExchange];
    __shared__ float sums[kRows][GL * 8 + 1];
    const int half = a.d / 2, heads = a.heads[0] + a.heads[1];
    const int wave = threadIdx.x / 64, lane = threadIdx.x % GL, grp = threadIdx.x % 64 / GL;
    const bool live = 8 * lane < a.d;
    const float inv_d = 1.0f / (float)a.d;
    float *exr = &ex[L == kInterleaved ? 0 : wave][L == kInterleaved ? 0 : grp * GL * 8];
    float dw0[8], dw1[8], w0[8], w1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dw0[i] = dw1[i] = 0.0f;
    load_weights(a.w[0], lane, live, w0);
    load_weights(a.w[1], lane, live, w1);
    const Steps st = steps_of<GL>(a);
    const auto load = [&](int64_t token, int head, u32x4 &xv, u32x4 &gv) {
        xv = gv = u32x4{0, 0, 0, 0};
        const int h = head + grp;
        if (h < heads && live) {
            const bool k = h >= a.heads[0];
            const int hh = k ? h - a.heads[0] : h;
            const Heads x = k ? a.x[1] : a.x[0], g = k ? g1 : g0;
            xv = *reinterpret_cast<const u32x4 *>(x.p + token * x.st + hh * x.sh + 8 * lane);
            gv = *reinterpret_cast<const u32x4 *>(g.p + token * g.st + hh * g.sh + 8 * lane);
        }
    };
    int64_t token = st.token;
    int head = st.head;
    Turn<L> turn;
    u32x4 nx = {0, 0, 0, 0}, ng = nx;
    if (st.begin < st.end) {
        load(token, head, nx, ng);
        turn.set(a.rope, token, half, lane, live, -1.0f, cs[wave]);
    }
    for (int64_t i = st.begin; i < st.end; ++i) {
        const u32x4 cx = nx, cg = ng;
        int64_t token2 = token;
        int head2 = head;
        next_step<GL>(a, token2, head2);
        if (i + 1 < st.end) load(token2, head2, nx, ng);
        const int h = head + grp;
        const bool k = h >= a.heads[0];
        float x[8], g[8];
        unpack8(cx, x);
        unpack8(cg, g);
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(x[e], x[e], sum);
        const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(head_sum<GL>(sum), inv_d, a.eps));
        const float rr = h < heads ? r : 0.0f;  // rows that are not there leave zeros in the sums, also with eps = 0
        turn.apply(g, lane, a.rope.pairs, exr);
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] *= rr;
            const float p = g[e] * x[e];  // zero in lanes and heads that are not there
            dw0[e] += k ? 0.0f : p;
            dw1[e] += k ? p : 0.0f;
            g[e] *= k ? w1[e] : w0[e];
            dot = __builtin_fmaf(g[e], x[e], dot);
        }
        dot = head_sum<GL>(dot) * inv_d;
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = r * (g[e] - x[e] * dot);
        if (h < heads && live) {
            const int hh = k ? h - a.heads[0] : h;
            const HeadsOut o = k ? o1 : o0;
            *reinterpret_cast<u32x4 *>(o.p + token * o.st + hh * o.sh + 8 * lane) = pack8(g);
        }
        if (token2 != token && i + 1 < st.end) turn.set(a.rope, token2, half, lane, live, -1.0f, cs[wave]);
        token = token2;
        head = head2;
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[threadIdx.x / GL][8 * lane + i] = which ? dw1[i] : dw0[i];
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += kThreads) {
            float s = 0.0f;
            for (int r = 0; r < kRows; ++r) s += sums[r][c];
            partial[((int64_t)blockIdx.x * 2 + which) * a.d + c] = s;
        }
    }
}

// dw[which][c] = sum over blocks of partial[block][which][c]: 8 columns a
// workgroup, 128 threads a column.
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float *__restrict__ partial, int blocks, int d, float *dw0,
                                                       float *dw1) {
    __shared__ float sums[128][9];
    const int c = threadIdx.x % 8, r = threadIdx.x / 8, col = blockIdx.x * 8 + c;  // 2 d is a multiple of 8
    float v[kBlocksBwd / 128];
#pragma unroll
    for (int i = 0; i < kBlocksBwd / 128; ++i)
        v[i] = r + 128 * i < blocks ? partial[(int64_t)(r + 128 * i) * 2 * d + col] : 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kBlocksBwd / 128; ++i) s += v[i];
    sums[r][c] = s;
    __syncthreads();
    for (int n = 64; n > 0; n /= 2) {
        if (r < n) sums[r][c] += sums[r + n][c];
        __syncthreads();
    }
    if (r == 0) {
        float *dw = col < d ? dw0 : dw1;
        if (dw) dw[col < d ? col : col - d] = sums[0][c];
    }
}

int lanes_of(int d) { return d <= 32 ? 4 : d <= 64 ? 8 : d <= 128 ? 16 : 32; }
Layout layout_of(const Rope &r) { return r.interleaved ? kInterleaved : r.pairs % 8 == 0 ? kHalves : kHalvesOdd; }

// Calls f(integral_constant lanes, integral_constant layout).
template <class F>
hipError_t dispatch(int lanes, Layout l, F f) {
    auto with = [&](auto gl) {
        if (l == kInterleaved) return f(gl, std::integral_constant<int, kInterleaved>{});
        if (l == kHalves) return f(gl, std::integral_constant<int, kHalves>{});
        return f(gl, std::integral_constant<int, kHalvesOdd>{});
    };
    if (lanes == 4) return with(std::integral_constant<int, 4>{});
    if (lanes == 8) return with(std::integral_constant<int, 8>{});
    if (lanes == 16) return with(std::integral_constant<int, 16>{});
    return with(std::integral_constant<int, 32>{});
}

// Steps of all tokens.
int64_t steps_of(const NormRope &a) {
    const int rows = 64 / lanes_of(a.d);
    return a.tokens * ((a.heads[0] + a.heads[1] + rows - 1) / rows);
}

}  // namespace

hipError_t launch_qk_norm_rope(const NormRope &a, const HeadsOut out[2], hipStream_t stream) {
    // as many wavefronts as the card holds at a time, fewer where there are fewer steps
    const int64_t blocks = (steps_of(a) + 3) / 4;
    const unsigned grid = (unsigned)(blocks < kBlocks ? blocks : kBlocks);
    return dispatch(lanes_of(a.d), layout_of(a.rope), [&](auto gl, auto l) {
        norm_rope_kernel<gl.value, l.value><<<dim3(grid), kThreads, 0, stream>>>(a, out[0], out[1]);
        return hipGetLastError();
    });
}

int64_t qk_norm_rope_blocks(int64_t) { return kBlocksBwd; }

hipError_t launch_qk_norm_rope_backward(const NormRope &a, const Heads dy[2], const HeadsOut dx[2], float *const dw[2],
                                        float *partial, hipStream_t stream) {
    const int64_t blocks = (steps_of(a) + 3) / 4;
    const unsigned grid = (unsigned)(blocks < kBlocksBwd ? blocks : kBlocksBwd);
    const hipError_t e = dispatch(lanes_of(a.d), layout_of(a.rope), [&](auto gl, auto l) {
        norm_rope_bwd_kernel<gl.value, l.value><<<dim3(grid), kThreads, 0, stream>>>(a, dy[0], dy[1], dx[0], dx[1], partial);
        return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    norm_dw_kernel<<<dim3((unsigned)(a.d / 4)), 1024, 0, stream>>>(partial, (int)grid, a.d, dw[0], dw[1]);
    return hipGetLastError();
}

}  // namespace ck4
