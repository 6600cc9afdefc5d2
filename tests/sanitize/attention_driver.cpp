// Host-only driver of the attention-block entry points' argument validation
// (tests/test_attention_sanitizers.py), built with the address and
// undefined-behaviour sanitizers. The launchers and the device check are
// stand-ins. Valid arguments launch once; arguments at the limits of their
// types are refused without overflow and launch nothing.
#include <climits>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "api_common.h"
#include "attn_kernels.h"
#include "ck4.h"

static int g_launches = 0, g_failures = 0;

namespace ck4 {
ck4_status api_fail(ck4_status s, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return s;
}
ck4_status api_check_device(const char *, int *) { return CK4_OK; }
ck4_status api_launched(const char *, hipError_t e) { return e == hipSuccess ? CK4_OK : CK4_ERR_DEVICE; }
hipError_t launch_qk_norm_rope(const NormRope &, const HeadsOut[2], hipStream_t) { return ++g_launches, hipSuccess; }
int64_t qk_norm_rope_blocks(int64_t tokens) { return tokens < 1024 ? tokens : 1024; }
hipError_t launch_qk_norm_rope_backward(const NormRope &, const Heads[2], const HeadsOut[2], float *const[2], float *,
                                        hipStream_t) { return ++g_launches, hipSuccess; }
int64_t attention_floats(int seqs, int64_t tq, int64_t tk, int hq, int d) { return (seqs + tq / 256 + tk / 64) * hq * d; }
int64_t attention_backward_floats(int seqs, int64_t tq, int64_t tk, int hq, int hk, int d) {
    return 2 * tq * hq + (seqs + tk / 256) * hk * d;
}
hipError_t launch_attention(const Attn &, const HeadsOut &, float *, float *, hipStream_t) {
    return ++g_launches, hipSuccess;
}
hipError_t launch_attention_backward(const Attn &, const Heads &, const Heads &, const float *, float *, const HeadsOut &,
                                     const HeadsOut &, const HeadsOut &, hipStream_t) { return ++g_launches, hipSuccess; }
int64_t attention_decode_floats(int64_t batch, int64_t, int hq, int hk, int d) { return (512 + batch * hq / hk) * 16 * (d + 2); }
hipError_t launch_attention_decode(const Decode &, float *, const HeadsOut &, float *, hipStream_t) {
    return ++g_launches, hipSuccess;
}
}  // namespace ck4

static void expect(const char *what, ck4_status got, bool valid) {
    const bool ok = valid ? got == CK4_OK && g_launches == 1 : got != CK4_OK && g_launches == 0;
    if (!ok) {
        std::printf("FAIL %s: status %d, %d launches\n", what, (int)got, g_launches);
        ++g_failures;
    }
    g_launches = 0;
}

int main() {
    auto *p = reinterpret_cast<uint16_t *>(static_cast<uintptr_t>(1) << 20);
    auto *f = reinterpret_cast<float *>(p);
    auto *n = reinterpret_cast<int32_t *>(p);
    const int64_t big[] = {INT64_MAX, INT64_MAX - 7, INT64_MIN, -8, INT64_C(1) << 62, INT64_C(1) << 41};
    const int bigi[] = {INT_MAX, INT_MAX - 7, INT_MIN, -8};

    auto norm = [&](int64_t st, int64_t sh, int64_t tokens, int h, int d, const int *secs) {
        return ck4_qk_norm_rope(p, st, sh, p, st, sh, tokens, h, h, d, f, f, n, 0, 4, secs, f, 1, 1e-6f, p, st, sh, p, st,
                                sh, nullptr);
    };
    auto norm_bwd = [&](int64_t st, int64_t sh, int64_t tokens, int h, int d, const int *secs) {
        return ck4_qk_norm_rope_backward(p, st, sh, p, st, sh, p, st, sh, p, st, sh, tokens, h, h, d, f, f, n, 0, 4, secs, f,
                                         1, 1e-6f, p, st, sh, p, st, sh, f, f, p, SIZE_MAX, nullptr);
    };
    auto attn = [&](int64_t st, int64_t sh, int64_t t, int h, int d, int64_t seqs) {
        return ck4_attention(p, st, sh, p, st, sh, p, st, sh, n, n, seqs, t, t, h, h, d, 1, 0.1f, p, st, sh, f, p, SIZE_MAX,
                             nullptr);
    };
    auto attn_bwd = [&](int64_t st, int64_t sh, int64_t t, int h, int d, int64_t seqs) {
        return ck4_attention_backward(p, st, sh, p, st, sh, p, st, sh, p, st, sh, p, st, sh, f, n, n, seqs, t, t, h, h, d, 1,
                                      0.1f, p, st, sh, p, st, sh, p, st, sh, p, SIZE_MAX, nullptr);
    };
    auto decode = [&](int64_t st, int64_t sh, int64_t t, int h, int d, int64_t sb) {
        return ck4_attention_decode(p, st, sh, p, sb, st, sh, p, sb, st, sh, n, t, t, h, h, d, 0.1f, p, st, sh, f, p,
                                    SIZE_MAX, nullptr);
    };
    const int secs[4] = {8, 8, 8, 8};
    expect("norm", norm(256, 64, 5, 4, 64, secs), true);
    expect("norm, one token and head", norm(INT64_MIN / 8 * 8, INT64_MIN / 8 * 8, 1, 1, 64, secs), true);
    const int none[4] = {0, 0, 0, 0};  // no pair is turned: no frequencies
    expect("norm without rotation", ck4_qk_norm_rope(p, 256, 64, p, 256, 64, 5, 4, 4, 64, f, f, n, 0, 4, none, nullptr, 1,
                                                     1e-6f, p, 256, 64, p, 256, 64, nullptr), true);
    expect("norm without frequencies", ck4_qk_norm_rope(p, 256, 64, p, 256, 64, 5, 4, 4, 64, f, f, n, 0, 4, secs, nullptr, 1,
                                                        1e-6f, p, 256, 64, p, 256, 64, nullptr), false);
    expect("norm_bwd", norm_bwd(256, 64, 5, 4, 64, secs), true);
    expect("attn", attn(256, 64, 5, 4, 64, 3), true);
    expect("attn, heads first", attn(64, 320, 5, 4, 64, 3), true);
    expect("attn_bwd", attn_bwd(256, 64, 5, 4, 64, 3), true);
    expect("decode", decode(256, 64, 5, 4, 64, 1280), true);
    expect("decode, the widest strides", decode(1 << 24, INT64_C(1) << 40, 5, 4, 64, INT64_C(1) << 40), true);
    for (int64_t b : big) {
        expect("norm st", norm(b, 64, 5, 4, 64, secs), false);
        expect("norm sh", norm(256, b, 5, 4, 64, secs), false);
        expect("norm tokens", norm(256, 64, b, 4, 64, secs), false);
        expect("norm_bwd st", norm_bwd(b, 64, 5, 4, 64, secs), false);
        expect("norm_bwd tokens", norm_bwd(256, 64, b, 4, 64, secs), false);
        expect("attn st", attn(b, 64, 5, 4, 64, 3), false);
        expect("attn sh", attn(256, b, 5, 4, 64, 3), false);
        expect("attn tokens", attn(256, 64, b, 4, 64, 3), false);
        expect("attn seqs", attn(256, 64, 5, 4, 64, b), false);
        expect("attn_bwd tokens", attn_bwd(256, 64, b, 4, 64, 3), false);
        expect("decode st", decode(b, 64, 5, 4, 64, 1280), false);
        expect("decode sb", decode(256, 64, 5, 4, 64, b), false);
        expect("decode batch", decode(256, 64, b, 4, 64, 1280), false);
        ck4_qk_norm_rope_workspace_bytes(b, 64);
        ck4_attention_workspace_bytes(b, b, b, 4, 4, 64);
        ck4_attention_backward_workspace_bytes(1, b, 4, 4, 4, 64);
        ck4_attention_backward_workspace_bytes(b, 4, b, 4, 4, 64);
        ck4_attention_decode_workspace_bytes(b, b, 4, 4, 64);
    }
    for (int b : bigi) {
        const int bad[4] = {8, b, b, 8};
        expect("norm heads", norm(256, 64, 5, b, 64, secs), false);
        expect("norm d", norm(256, 64, 5, 4, b, secs), false);
        expect("norm sections", norm(256, 64, 5, 4, 64, bad), false);
        expect("attn heads", attn(256, 64, 5, b, 64, 3), false);
        expect("attn d", attn(256, 64, 5, 4, b, 3), false);
        expect("decode heads", decode(256, 64, 5, b, 64, 1280), false);
        ck4_qk_norm_rope_workspace_bytes(4, b);
        ck4_attention_workspace_bytes(1, 4, 4, b, b, 64);
        ck4_attention_backward_workspace_bytes(1, 4, 4, 4, b, 64);
        ck4_attention_backward_workspace_bytes(1, 4, 4, 4, 4, b);
        ck4_attention_decode_workspace_bytes(4, 4, b, 4, 64);
        ck4_attention_decode_workspace_bytes(4, 4, 4, b, 64);
    }
    std::printf("%d failures\n", g_failures);
    return g_failures != 0;
}
