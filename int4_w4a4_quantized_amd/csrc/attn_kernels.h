// Internal launchers of the attention-block kernels (gfx950): head norm with
// rotary positions, attention over packed sequences, their gradients, and
// attention of single tokens over a cache. Not part of the C ABI:
// attention_api.cpp validates arguments and then calls these.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ck4 {

// bf16 heads [tokens, heads, d]: element (t, h, c) at p[t * st + h * sh + c].
// Strides in elements, multiples of 8; p 16-byte aligned; d a multiple of 8.
struct Heads {
    const uint16_t *p;
    int64_t st, sh;
};
struct HeadsOut {
    uint16_t *p;
    int64_t st, sh;
};

constexpr int kMaxAxes = 4;

// Rotary positions: pair j of a head turns by position(axis of j) * freqs[j].
// Axis a owns the pairs [end[a - 1], end[a]).
struct Rope {
    const void *pos;     // [tokens, axes], int32 or fp32
    const float *freqs;  // [pairs]
    int end[kMaxAxes];
    int axes;
    int pairs;           // rotated elements / 2
    bool pos_f32;
    bool interleaved;    // pairs (2j, 2j + 1), else (j, j + pairs)
};

// The two head groups of one call share tokens, head size and rotation, and
// have a norm weight (fp32 [d], or null: ones) each.
struct NormRope {
    Heads x[2];
    const float *w[2];
    int heads[2];
    int64_t tokens;
    int d;
    float eps;
    Rope rope;
};

hipError_t launch_qk_norm_rope(const NormRope &a, const HeadsOut out[2], hipStream_t stream);

// Row blocks of the backward kernel: the partial weight gradients take
// blocks * 2 * d floats of workspace.
int64_t qk_norm_rope_blocks(int64_t tokens);
hipError_t launch_qk_norm_rope_backward(const NormRope &a, const Heads dy[2], const HeadsOut dx[2], float *const dw[2],
                                        float *partial, hipStream_t stream);

// Packed sequences: sequence i owns rows [cu[i], cu[i + 1]) of its tensor,
// cu int32 [seqs + 1] on the device (null: one sequence of all rows). The
// kernels clamp what they read from cu to [0, rows], and cut tiles only where
// the steps that they count fit what the workspace was sized for, so no content
// makes them leave the tensors or the workspace.
struct Packed {
    const int32_t *cu_q, *cu_k;
    int64_t tq, tk;
    int seqs;
};

struct Attn {
    Heads q, k, v;
    Packed rows;
    int hq, hk, d;
    bool causal;
    float scale;
};

// Floats of workspace of the two calls (the first may be 0).
int64_t attention_floats(int seqs, int64_t tq, int64_t tk, int hq, int d);
int64_t attention_backward_floats(int seqs, int64_t tq, int64_t tk, int hq, int hk, int d);

hipError_t launch_attention(const Attn &a, const HeadsOut &out, float *lse, float *workspace, hipStream_t stream);
hipError_t launch_attention_backward(const Attn &a, const Heads &out, const Heads &dout, const float *lse, float *workspace,
                                     const HeadsOut &dq, const HeadsOut &dk, const HeadsOut &dv, hipStream_t stream);

// One query token per sequence over a cache: element (b, slot, head, c) of
// k at k.p[b * k_sb + slot * k.st + head * k.sh + c]; lengths int32 [batch] on
// the device, clamped to [0, slots].
struct Decode {
    Heads q;             // [batch, hq, d]
    Heads k, v;
    int64_t k_sb, v_sb;
    const int32_t *lengths;
    int64_t batch, slots;
    int hq, hk, d;
    float scale;
};

// The floats of workspace that the workgroups' partial results take.
int64_t attention_decode_floats(int64_t batch, int64_t slots, int hq, int hk, int d);  // may be 0
hipError_t launch_attention_decode(const Decode &a, float *partial, const HeadsOut &out, float *lse, hipStream_t stream);

}  // namespace ck4
