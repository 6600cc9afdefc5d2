// C ABI of the attention-block operators: argument validation, launch
// selection, errors. Every entry point validates everything before it touches
// the device, so a rejected call launches nothing.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/ck4.h"
#include "api_common.h"
#include "attn_kernels.h"

using ck4::api_fail;

namespace {

constexpr int64_t kMaxTokens = INT64_C(1) << 30;
constexpr int kMaxHeads = 4096;
// Strides: one 64-row tile stays within the 4 GiB that a buffer descriptor spans.
constexpr int64_t kMaxRowStride = INT64_C(1) << 24;
// ... and element offsets (tokens * stride + heads * stride) stay far inside int64.
constexpr int64_t kMaxHeadStride = INT64_C(1) << 40;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Strides of a [tokens, heads, d] tensor; one that steps over a dimension of size 1 is not looked at (d stands for it).
ck4_status check_heads(const char *fn, const char *name, const void *p, int64_t tokens, int heads, int d, int64_t *st,
                       int64_t *sh, bool written) {
    if (tokens == 1) *st = d;
    if (heads == 1) *sh = d;
    if (!aligned(p, 16)) return api_fail(CK4_ERR_INVALID, "%s: %s not 16-byte aligned", fn, name);
    if (*st % 8 || *sh % 8) return api_fail(CK4_ERR_INVALID, "%s: strides of %s are not multiples of 8", fn, name);
    if ((tokens > 1 && *st < d) || (heads > 1 && *sh < d))
        return api_fail(CK4_ERR_INVALID, "%s: a stride of %s is smaller than a head", fn, name);
    if (*st > kMaxRowStride || *sh > kMaxHeadStride)
        return api_fail(CK4_ERR_UNSUPPORTED, "%s: a stride of %s is too large", fn, name);
    // rows of an output must not overlap: whole tokens inside a head's step, or whole heads inside a token's
    if (written && tokens > 1 && heads > 1 && *st < (heads - 1) * *sh + d && *sh < (tokens - 1) * *st + d)
        return api_fail(CK4_ERR_INVALID, "%s: the heads of %s overlap", fn, name);
    return CK4_OK;
}

// The kernels stand in for "no score yet" with -1e30, which times scale must stay finite.
ck4_status check_scale(const char *fn, float scale) {
    if (!(scale > 0.0f) || !std::isfinite(scale)) return api_fail(CK4_ERR_INVALID, "%s: scale=%g", fn, (double)scale);
    if (scale > 1e6f) return api_fail(CK4_ERR_UNSUPPORTED, "%s: scale=%g > 1e6", fn, (double)scale);
    return CK4_OK;
}

ck4_status check_norm_rope(const char *fn, int64_t tokens, int hq, int hk, int d, const void *q, const void *k,
                           const float *q_weight, const float *k_weight, const void *positions, int axes,
                           const int *sections, const float *freqs, float eps, ck4::NormRope *a) {
    if (!q || !k || !positions || !sections) return api_fail(CK4_ERR_INVALID, "%s: null pointer", fn);
    if (tokens <= 0 || hq <= 0 || hk <= 0 || d <= 0)
        return api_fail(CK4_ERR_INVALID, "%s: tokens, hq, hk and d must be positive", fn);
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return api_fail(CK4_ERR_INVALID, "%s: eps=%g", fn, (double)eps);
    if (d % 8 != 0 || d > 256)
        return api_fail(CK4_ERR_UNSUPPORTED, "%s: d=%d (need a multiple of 8 up to 256)", fn, d);
    if (tokens > kMaxTokens || hq > kMaxHeads || hk > kMaxHeads)
        return api_fail(CK4_ERR_UNSUPPORTED, "%s: too many tokens or heads", fn);
    if (axes < 1 || axes > ck4::kMaxAxes)
        return api_fail(CK4_ERR_UNSUPPORTED, "%s: axes=%d (need 1 to %d)", fn, axes, ck4::kMaxAxes);
    int pairs = 0;
    for (int i = 0; i < ck4::kMaxAxes; ++i) {
        if (i < axes) {
            if (sections[i] < 0 || sections[i] > d / 2 - pairs)
                return api_fail(CK4_ERR_INVALID, "%s: sections[%d]=%d: the sections hold at most d / 2 = %d pairs", fn, i,
                                sections[i], d / 2);
            pairs += sections[i];
        }
        a->rope.end[i] = pairs;
    }
    if (pairs > 0 && !freqs) return api_fail(CK4_ERR_INVALID, "%s: null pointer", fn);
    if (!aligned(positions, 4) || !aligned(freqs, 4) || !aligned(q_weight, 4) || !aligned(k_weight, 4))
        return api_fail(CK4_ERR_INVALID, "%s: positions, freqs or a weight not 4-byte aligned", fn);
    a->tokens = tokens;
    a->heads[0] = hq;
    a->heads[1] = hk;
    a->d = d;
    a->eps = eps;
    a->w[0] = q_weight;
    a->w[1] = k_weight;
    a->rope.pos = positions;
    a->rope.freqs = freqs;
    a->rope.axes = axes;
    a->rope.pairs = pairs;
    return CK4_OK;
}

}  // namespace

extern "C" {

ck4_status ck4_qk_norm_rope(const uint16_t *q, int64_t q_st, int64_t q_sh, const uint16_t *k, int64_t k_st, int64_t k_sh,
                            int64_t tokens, int hq, int hk, int d, const float *q_weight, const float *k_weight,
                            const void *positions, int positions_f32, int axes, const int *sections, const float *freqs,
                            int interleaved, float eps, uint16_t *q_out, int64_t qo_st, int64_t qo_sh, uint16_t *k_out,
                            int64_t ko_st, int64_t ko_sh, void *stream) {
    const char *fn = "ck4_qk_norm_rope";
    ck4::NormRope a{};
    if (!q_out || !k_out) return api_fail(CK4_ERR_INVALID, "%s: null pointer", fn);
    if (ck4_status s = check_norm_rope(fn, tokens, hq, hk, d, q, k, q_weight, k_weight, positions, axes, sections, freqs,
                                       eps, &a))
        return s;
    if (ck4_status s = check_heads(fn, "q", q, tokens, hq, d, &q_st, &q_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "k", k, tokens, hk, d, &k_st, &k_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "q_out", q_out, tokens, hq, d, &qo_st, &qo_sh, true)) return s;
    if (ck4_status s = check_heads(fn, "k_out", k_out, tokens, hk, d, &ko_st, &ko_sh, true)) return s;
    if (ck4_status s = ck4::api_check_device(fn, nullptr)) return s;
    a.x[0] = {q, q_st, q_sh};
    a.x[1] = {k, k_st, k_sh};
    a.rope.pos_f32 = positions_f32 != 0;
    a.rope.interleaved = interleaved != 0;
    const ck4::HeadsOut out[2] = {{q_out, qo_st, qo_sh}, {k_out, ko_st, ko_sh}};
    return ck4::api_launched(fn, ck4::launch_qk_norm_rope(a, out, static_cast<hipStream_t>(stream)));
}

size_t ck4_qk_norm_rope_workspace_bytes(int64_t tokens, int d) {
    if (tokens <= 0 || tokens > kMaxTokens || d <= 0 || d % 8 != 0 || d > 256) return 0;
    return (size_t)ck4::qk_norm_rope_blocks(tokens) * 2 * d * sizeof(float);
}

ck4_status ck4_qk_norm_rope_backward(const uint16_t *dq_out, int64_t dqo_st, int64_t dqo_sh, const uint16_t *dk_out,
                                     int64_t dko_st, int64_t dko_sh, const uint16_t *q, int64_t q_st, int64_t q_sh,
                                     const uint16_t *k, int64_t k_st, int64_t k_sh, int64_t tokens, int hq, int hk, int d,
                                     const float *q_weight, const float *k_weight, const void *positions,
                                     int positions_f32, int axes, const int *sections, const float *freqs,
                                     int interleaved, float eps, uint16_t *dq, int64_t dq_st, int64_t dq_sh, uint16_t *dk,
                                     int64_t dk_st, int64_t dk_sh, float *dq_weight, float *dk_weight, void *workspace,
                                     size_t ws_bytes, void *stream) {
    const char *fn = "ck4_qk_norm_rope_backward";
    ck4::NormRope a{};
    if (!dq_out || !dk_out || !dq || !dk) return api_fail(CK4_ERR_INVALID, "%s: null pointer", fn);
    if (ck4_status s = check_norm_rope(fn, tokens, hq, hk, d, q, k, q_weight, k_weight, positions, axes, sections, freqs,
                                       eps, &a))
        return s;
    if (ck4_status s = check_heads(fn, "dq_out", dq_out, tokens, hq, d, &dqo_st, &dqo_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "dk_out", dk_out, tokens, hk, d, &dko_st, &dko_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "q", q, tokens, hq, d, &q_st, &q_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "k", k, tokens, hk, d, &k_st, &k_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "dq", dq, tokens, hq, d, &dq_st, &dq_sh, true)) return s;
    if (ck4_status s = check_heads(fn, "dk", dk, tokens, hk, d, &dk_st, &dk_sh, true)) return s;
    if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4) || !aligned(workspace, 4))
        return api_fail(CK4_ERR_INVALID, "%s: dq_weight, dk_weight or workspace not 4-byte aligned", fn);
    const size_t need = ck4_qk_norm_rope_workspace_bytes(tokens, d);
    if (!workspace || ws_bytes < need)
        return api_fail(CK4_ERR_INVALID, "%s: workspace %zu bytes < %zu needed", fn, workspace ? ws_bytes : 0, need);
    if (ck4_status s = ck4::api_check_device(fn, nullptr)) return s;
    a.x[0] = {q, q_st, q_sh};
    a.x[1] = {k, k_st, k_sh};
    a.rope.pos_f32 = positions_f32 != 0;
    a.rope.interleaved = interleaved != 0;
    const ck4::Heads dy[2] = {{dq_out, dqo_st, dqo_sh}, {dk_out, dko_st, dko_sh}};
    const ck4::HeadsOut dx[2] = {{dq, dq_st, dq_sh}, {dk, dk_st, dk_sh}};
    float *const dw[2] = {dq_weight, dk_weight};
    return ck4::api_launched(fn, ck4::launch_qk_norm_rope_backward(a, dy, dx, dw, static_cast<float *>(workspace),
                                                                   static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// The kernels count tiles of 256 rows per head, and steps of 64, in 32 bits: so many of 64, and a part tile of queries
// and one of keys per sequence, are more than one launch takes.
bool too_many_tiles(int64_t seqs, int64_t tq, int64_t tk, int hq) {
    return (tq / 64 + tk / 64 + 2 * seqs + 2) * hq > INT32_MAX / 2;
}

// Shapes, strides and options that the attention calls share.
ck4_status check_attention(const char *fn, const uint16_t *q, int64_t *q_st, int64_t *q_sh, const uint16_t *k,
                           int64_t *k_st, int64_t *k_sh, const uint16_t *v, int64_t *v_st, int64_t *v_sh,
                           const int32_t *cu_q, const int32_t *cu_k, int64_t seqs, int64_t tq, int64_t tk, int hq, int hk,
                           int d, int causal, float scale, ck4::Attn *a) {
    if (!q || !k || !v) return api_fail(CK4_ERR_INVALID, "%s: null pointer", fn);
    if (tq <= 0 || tk <= 0 || hq <= 0 || hk <= 0 || d <= 0 || seqs <= 0)
        return api_fail(CK4_ERR_INVALID, "%s: tq, tk, hq, hk, d and seqs must be positive", fn);
    if ((cu_q == nullptr) != (cu_k == nullptr) || (!cu_q && seqs != 1))
        return api_fail(CK4_ERR_INVALID, "%s: cu_q and cu_k come together, or neither and seqs = 1", fn);
    if (!aligned(cu_q, 4) || !aligned(cu_k, 4)) return api_fail(CK4_ERR_INVALID, "%s: cu_q or cu_k misaligned", fn);
    if (ck4_status s = check_scale(fn, scale)) return s;
    if (hq % hk != 0) return api_fail(CK4_ERR_INVALID, "%s: hq=%d is not a multiple of hk=%d", fn, hq, hk);
    if (d % 8 != 0 || d > 128)
        return api_fail(CK4_ERR_UNSUPPORTED, "%s: d=%d (need a multiple of 8 up to 128)", fn, d);
    if (tq > kMaxTokens || tk > kMaxTokens || hq > kMaxHeads || seqs > (1 << 20))
        return api_fail(CK4_ERR_UNSUPPORTED, "%s: too many tokens, heads or sequences", fn);
    if (too_many_tiles(seqs, tq, tk, hq))
        return api_fail(CK4_ERR_UNSUPPORTED, "%s: too many tiles for one launch", fn);
    if (ck4_status s = check_heads(fn, "q", q, tq, hq, d, q_st, q_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "k", k, tk, hk, d, k_st, k_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "v", v, tk, hk, d, v_st, v_sh, false)) return s;
    a->q = {q, *q_st, *q_sh};
    a->k = {k, *k_st, *k_sh};
    a->v = {v, *v_st, *v_sh};
    a->rows = {cu_q, cu_k, tq, tk, (int)seqs};
    a->hq = hq;
    a->hk = hk;
    a->d = d;
    a->causal = causal != 0;
    a->scale = scale;
    return CK4_OK;
}

// Whether the sizes are ones that a workspace size is given for (the calls check them again).
bool attention_sizes(int64_t seqs, int64_t tq, int64_t tk, int hq, int hk, int d) {
    return seqs > 0 && seqs <= (1 << 20) && tq > 0 && tq <= kMaxTokens && tk > 0 && tk <= kMaxTokens && hq > 0 &&
           hq <= kMaxHeads && hk > 0 && hq % hk == 0 && d > 0 && d % 8 == 0 && d <= 128 &&
           !too_many_tiles(seqs, tq, tk, hq);
}

}  // namespace

extern "C" {

size_t ck4_attention_workspace_bytes(int64_t seqs, int64_t tq, int64_t tk, int hq, int hk, int d) {
    if (!attention_sizes(seqs, tq, tk, hq, hk, d)) return 0;
    return (size_t)ck4::attention_floats((int)seqs, tq, tk, hq, d) * sizeof(float);
}

ck4_status ck4_attention(const uint16_t *q, int64_t q_st, int64_t q_sh, const uint16_t *k, int64_t k_st, int64_t k_sh,
                         const uint16_t *v, int64_t v_st, int64_t v_sh, const int32_t *cu_q, const int32_t *cu_k,
                         int64_t seqs, int64_t tq, int64_t tk, int hq, int hk, int d, int causal, float scale,
                         uint16_t *out, int64_t o_st, int64_t o_sh, float *lse, void *workspace, size_t ws_bytes,
                         void *stream) {
    const char *fn = "ck4_attention";
    ck4::Attn a{};
    if (!out) return api_fail(CK4_ERR_INVALID, "%s: null pointer", fn);
    if (ck4_status s = check_attention(fn, q, &q_st, &q_sh, k, &k_st, &k_sh, v, &v_st, &v_sh, cu_q, cu_k, seqs, tq, tk, hq,
                                       hk, d, causal, scale, &a))
        return s;
    if (ck4_status s = check_heads(fn, "out", out, tq, hq, d, &o_st, &o_sh, true)) return s;
    if (!aligned(lse, 4) || !aligned(workspace, 16))
        return api_fail(CK4_ERR_INVALID, "%s: lse or workspace misaligned", fn);
    const size_t need = ck4_attention_workspace_bytes(seqs, tq, tk, hq, hk, d);
    if (need > 0 && (!workspace || ws_bytes < need))
        return api_fail(CK4_ERR_INVALID, "%s: workspace %zu bytes < %zu needed", fn, workspace ? ws_bytes : 0, need);
    if (ck4_status s = ck4::api_check_device(fn, nullptr)) return s;
    return ck4::api_launched(fn, ck4::launch_attention(a, {out, o_st, o_sh}, lse, static_cast<float *>(workspace),
                                                       static_cast<hipStream_t>(stream)));
}

size_t ck4_attention_backward_workspace_bytes(int64_t seqs, int64_t tq, int64_t tk, int hq, int hk, int d) {
    if (!attention_sizes(seqs, tq, tk, hq, hk, d)) return 0;
    return (size_t)ck4::attention_backward_floats((int)seqs, tq, tk, hq, hk, d) * sizeof(float);
}

ck4_status ck4_attention_backward(const uint16_t *dout, int64_t do_st, int64_t do_sh, const uint16_t *q, int64_t q_st,
                                  int64_t q_sh, const uint16_t *k, int64_t k_st, int64_t k_sh, const uint16_t *v,
                                  int64_t v_st, int64_t v_sh, const uint16_t *out, int64_t o_st, int64_t o_sh,
                                  const float *lse, const int32_t *cu_q, const int32_t *cu_k, int64_t seqs, int64_t tq,
                                  int64_t tk, int hq, int hk, int d, int causal, float scale, uint16_t *dq, int64_t dq_st,
                                  int64_t dq_sh, uint16_t *dk, int64_t dk_st, int64_t dk_sh, uint16_t *dv, int64_t dv_st,
                                  int64_t dv_sh, void *workspace, size_t ws_bytes, void *stream) {
    const char *fn = "ck4_attention_backward";
    ck4::Attn a{};
    if (!dout || !out || !lse || !dq || !dk || !dv)
        return api_fail(CK4_ERR_INVALID, "%s: null pointer", fn);
    if (ck4_status s = check_attention(fn, q, &q_st, &q_sh, k, &k_st, &k_sh, v, &v_st, &v_sh, cu_q, cu_k, seqs, tq, tk, hq,
                                       hk, d, causal, scale, &a))
        return s;
    if (ck4_status s = check_heads(fn, "dout", dout, tq, hq, d, &do_st, &do_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "out", out, tq, hq, d, &o_st, &o_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "dq", dq, tq, hq, d, &dq_st, &dq_sh, true)) return s;
    if (ck4_status s = check_heads(fn, "dk", dk, tk, hk, d, &dk_st, &dk_sh, true)) return s;
    if (ck4_status s = check_heads(fn, "dv", dv, tk, hk, d, &dv_st, &dv_sh, true)) return s;
    if (!aligned(lse, 4) || !aligned(workspace, 16))
        return api_fail(CK4_ERR_INVALID, "%s: lse or workspace misaligned", fn);
    const size_t need = ck4_attention_backward_workspace_bytes(seqs, tq, tk, hq, hk, d);
    if (!workspace || ws_bytes < need)
        return api_fail(CK4_ERR_INVALID, "%s: workspace %zu bytes < %zu needed", fn, workspace ? ws_bytes : 0, need);
    if (ck4_status s = ck4::api_check_device(fn, nullptr)) return s;
    return ck4::api_launched(
        fn, ck4::launch_attention_backward(a, {out, o_st, o_sh}, {dout, do_st, do_sh}, lse, static_cast<float *>(workspace),
                                           {dq, dq_st, dq_sh}, {dk, dk_st, dk_sh}, {dv, dv_st, dv_sh},
                                           static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

// A batch stride is free (it may be smaller than the slots' extent where caches interleave), but it is a multiple of 8.
ck4_status check_batch_stride(const char *fn, const char *name, int64_t batch, int64_t *sb) {
    if (batch == 1) *sb = 0;
    if (*sb < 0 || *sb % 8)
        return api_fail(CK4_ERR_INVALID, "%s: the batch stride of %s is negative or not a multiple of 8", fn, name);
    if (*sb > kMaxHeadStride) return api_fail(CK4_ERR_UNSUPPORTED, "%s: the batch stride of %s is too large", fn, name);
    return CK4_OK;
}

// The kernels count query heads, and tiles of 32 slots per sequence and key head (or 16 query heads), in 32 bits.
bool decode_too_large(int64_t batch, int64_t slots, int hq, int hk) {
    return batch > (1 << 20) || slots > kMaxTokens || hq > kMaxHeads || batch * hq > INT32_MAX ||
           batch * (hk + hq / 16 + 1) * (slots / 32 + 1) > INT32_MAX / 2;
}

}  // namespace

extern "C" {

size_t ck4_attention_decode_workspace_bytes(int64_t batch, int64_t slots, int hq, int hk, int d) {
    if (batch <= 0 || slots <= 0 || hq <= 0 || hk <= 0 || hq % hk != 0 || d <= 0 || d % 8 != 0 || d > 128 ||
        decode_too_large(batch, slots, hq, hk))
        return 0;
    return (size_t)ck4::attention_decode_floats(batch, slots, hq, hk, d) * sizeof(float);
}

ck4_status ck4_attention_decode(const uint16_t *q, int64_t q_st, int64_t q_sh, const uint16_t *k, int64_t k_sb,
                                int64_t k_st, int64_t k_sh, const uint16_t *v, int64_t v_sb, int64_t v_st, int64_t v_sh,
                                const int32_t *lengths, int64_t batch, int64_t slots, int hq, int hk, int d, float scale,
                                uint16_t *out, int64_t o_st, int64_t o_sh, float *lse, void *workspace, size_t ws_bytes,
                                void *stream) {
    const char *fn = "ck4_attention_decode";
    if (!q || !k || !v || !lengths || !out) return api_fail(CK4_ERR_INVALID, "%s: null pointer", fn);
    if (batch <= 0 || slots <= 0 || hq <= 0 || hk <= 0 || d <= 0)
        return api_fail(CK4_ERR_INVALID, "%s: batch, slots, hq, hk and d must be positive", fn);
    if (ck4_status s = check_scale(fn, scale)) return s;
    if (hq % hk != 0) return api_fail(CK4_ERR_INVALID, "%s: hq=%d is not a multiple of hk=%d", fn, hq, hk);
    if (d % 8 != 0 || d > 128)
        return api_fail(CK4_ERR_UNSUPPORTED, "%s: d=%d (need a multiple of 8 up to 128)", fn, d);
    if (decode_too_large(batch, slots, hq, hk))
        return api_fail(CK4_ERR_UNSUPPORTED, "%s: batch, slots or heads too large", fn);
    if (ck4_status s = check_heads(fn, "q", q, batch, hq, d, &q_st, &q_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "k", k, slots, hk, d, &k_st, &k_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "v", v, slots, hk, d, &v_st, &v_sh, false)) return s;
    if (ck4_status s = check_heads(fn, "out", out, batch, hq, d, &o_st, &o_sh, true)) return s;
    if (ck4_status s = check_batch_stride(fn, "k", batch, &k_sb)) return s;
    if (ck4_status s = check_batch_stride(fn, "v", batch, &v_sb)) return s;
    if (!aligned(lengths, 4) || !aligned(lse, 4) || !aligned(workspace, 16))
        return api_fail(CK4_ERR_INVALID, "%s: lengths, lse or workspace misaligned", fn);
    const size_t need = ck4_attention_decode_workspace_bytes(batch, slots, hq, hk, d);
    if (need > 0 && (!workspace || ws_bytes < need))
        return api_fail(CK4_ERR_INVALID, "%s: workspace %zu bytes < %zu needed", fn, workspace ? ws_bytes : 0, need);
    if (ck4_status s = ck4::api_check_device(fn, nullptr)) return s;
    const ck4::Decode a{{q, q_st, q_sh}, {k, k_st, k_sh}, {v, v_st, v_sh}, k_sb, v_sb, lengths, batch, slots, hq, hk, d,
                        scale};
    return ck4::api_launched(fn, ck4::launch_attention_decode(a, static_cast<float *>(workspace), {out, o_st, o_sh}, lse,
                                                              static_cast<hipStream_t>(stream)));
}

}  // extern "C"
