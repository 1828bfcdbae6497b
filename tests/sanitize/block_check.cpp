// Drives the host side of the operators around the state layer (kda_block_api.cpp)
// with calls that are refused or have nothing to do, and its size arithmetic at
// the limits.  Nothing is launched.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "kda.h"

static int bad = 0;
static void expect(int got, int want, const char* what) {
    if (got != want) {
        printf("%s: status %d, expected %d (%s)\n", what, got, want, kda_last_error());
        ++bad;
    }
}

int main() {
    void* const p = reinterpret_cast<void*>(uintptr_t(0x7f0000000000));
    float* const f = static_cast<float*>(p);
    const int32_t* cu = static_cast<const int32_t*>(p);
    const int64_t far = 0x7fff0000;
    size_t n = 0;

    kda_scan_dims_t s = {};
    s.num_seqs = 3; s.channels = 1 << 20; s.total_tokens = far; s.dtype = KDA_BF16;
    expect(kda_scan_workspace_size(&s, 1, &n), KDA_OK, "scan size");
    if (n < (size_t)far / 128 * (1 << 20) * 8) ++bad;
    expect(kda_scan_fwd(&s, p, f, nullptr, cu, p, nullptr, nullptr, p, 256, nullptr), KDA_ERR_INVALID_ARGUMENT, "scan small");
    expect(kda_scan_fwd(&s, p, f, nullptr, cu, p, nullptr, nullptr, p, n, nullptr), KDA_ERR_INVALID_ARGUMENT, "scan large");
    expect(kda_scan_bwd(&s, p, f, nullptr, cu, nullptr, p, nullptr, p, f, nullptr, p, n, nullptr), KDA_ERR_INVALID_ARGUMENT,
           "scan gradient large");
    s.total_tokens = 3; s.num_seqs = 3; s.x_stride = INT64_MIN;
    expect(kda_scan_step(&s, p, f, f, f, p, nullptr), KDA_ERR_INVALID_ARGUMENT, "scan step stride");
    s.x_stride = 0; s.num_seqs = 0; s.total_tokens = 0;
    expect(kda_scan_step(&s, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr), KDA_OK, "scan step empty");
    expect(kda_scan_bwd(&s, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                        nullptr, 0, nullptr), KDA_OK, "scan gradient empty");

    kda_conv_dims_t c = {};
    c.num_seqs = 1 << 30; c.channels = 1 << 20; c.total_tokens = far; c.dtype = KDA_F32; c.width = 4; c.activation = KDA_ACT_SILU;
    expect(kda_conv_bwd_workspace_size(&c, &n), KDA_OK, "conv size");
    expect(kda_conv_bwd(&c, p, f, f, p, cu, p, p, p, f, f, nullptr, p, 0, nullptr), KDA_ERR_INVALID_ARGUMENT, "conv small");
    c.num_seqs = INT32_MIN;
    expect(kda_conv_fwd(&c, p, f, f, p, cu, p, nullptr, nullptr), KDA_ERR_INVALID_ARGUMENT, "conv seqs");
    c.num_seqs = 0; c.total_tokens = 0;
    expect(kda_conv_step(&c, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr), KDA_OK, "conv step empty");

    kda_norm_gate_dims_t g = {};
    g.tokens = INT64_MAX; g.heads = INT32_MAX; g.width = 8192; g.dtype = KDA_BF16; g.activation = KDA_ACT_SILU; g.eps = 1e-6f;
    expect(kda_norm_gate_fwd(&g, p, f, p, p, nullptr), KDA_ERR_INVALID_ARGUMENT, "norm rows");
    g.tokens = far; g.heads = 1;
    expect(kda_norm_gate_bwd_workspace_size(&g, &n), KDA_OK, "norm size");
    expect(kda_norm_gate_bwd(&g, p, f, p, p, p, p, f, nullptr, 0, nullptr), KDA_ERR_INVALID_ARGUMENT, "norm workspace");
    g.tokens = 0;
    expect(kda_norm_gate_fwd(&g, nullptr, nullptr, nullptr, nullptr, nullptr), KDA_OK, "norm empty");

    kda_residual_norm_dims_t r = {};
    r.tokens = far; r.width = 8192; r.dtype = KDA_BF16; r.residual_dtype = KDA_F32; r.eps = 0.f; r.scale = 1.f;
    expect(kda_residual_norm_bwd_workspace_size(&r, &n), KDA_OK, "residual size");
    expect(kda_residual_norm_bwd(&r, p, p, f, f, p, p, p, p, f, f, p, n - 1, nullptr), KDA_ERR_INVALID_ARGUMENT, "residual small");
    r.dresidual_stride = 8191;
    expect(kda_residual_norm_fwd(&r, p, p, f, f, p, p, nullptr), KDA_ERR_INVALID_ARGUMENT, "residual stride");

    if (bad) return 1;
    printf("block api sanitizer check ok\n");
    return 0;
}
