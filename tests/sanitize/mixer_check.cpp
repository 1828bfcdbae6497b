// Drives the host side of the state space scan, the gated feed-forward products and
// the state cache with calls that are refused or have nothing to do, and their size
// arithmetic at the limits.  Nothing is launched.
#include <stdint.h>
#include <stdio.h>

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

    const int32_t shapes[][4] = {{1, 1, 1, 1}, {65536, 1, 256, 8192}, {65536, 65536, 256, 8192}, {65536, 256, 1, 1},
                                 {7, 7, 255, 33}, {96, 8, 128, 64}};
    for (auto& s : shapes)
        for (int32_t dt = 0; dt < 2; ++dt)
            for (int64_t t : {(int64_t)0, (int64_t)1, (int64_t)65, (int64_t)1 << 20, far})
                for (int32_t seqs : {1, 3, 1 << 20, (int)far})
                    for (int back = 0; back < 2; ++back) {
                        kda_ssm_dims_t d = {};
                        d.num_seqs = seqs; d.total_tokens = t; d.heads = s[0]; d.groups = s[1]; d.state = s[2]; d.width = s[3];
                        d.dtype = dt;
                        n = 0;
                        const int got = kda_ssm_workspace_size(&d, back, &n);
                        if (got == KDA_OK && back && n < (uint64_t)t / 64 * s[0] * s[2] * s[3] * 8) ++bad;
                        if (got == KDA_OK && n > 256 && back)
                            expect(kda_ssm_bwd(&d, p, f, f, p, p, f, f, f, cu, p, f, p, f, f, p, p, f, f, nullptr, p, 255,
                                               nullptr), KDA_ERR_INVALID_ARGUMENT, "scan gradient small");
                        d.num_seqs = (int32_t)(t < far ? t : far);
                        kda_ssm_conv_step_workspace_size(&d, &n);
                    }
    kda_ssm_dims_t s = {};
    s.heads = 2; s.groups = 1; s.state = 16; s.width = 16; s.dtype = KDA_BF16;
    s.num_seqs = 2; s.total_tokens = 2; s.x_stride = INT64_MIN;
    expect(kda_ssm_step(&s, p, f, f, p, p, f, f, f, f, p, nullptr), KDA_ERR_INVALID_ARGUMENT, "step stride");
    s.x_stride = 0; s.num_seqs = INT32_MIN;
    expect(kda_ssm_fwd(&s, p, f, f, p, p, f, f, f, cu, p, nullptr, nullptr, 0, nullptr), KDA_ERR_INVALID_ARGUMENT, "seqs");
    s.num_seqs = 0; s.total_tokens = 0;
    expect(kda_ssm_fwd(&s, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                       nullptr, nullptr, 0, nullptr), KDA_OK, "scan empty");
    expect(kda_ssm_conv_step(&s, 4, KDA_ACT_SILU, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                             nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr), KDA_OK, "conv step empty");

    const int32_t sizes[][2] = {{1, 1}, {1 << 20, 1 << 20}, {1 << 20, 1}, {1, 1 << 20}, {4096, 10240}, {1000, 2731}};
    for (auto& z : sizes)
        for (int32_t dt = 0; dt < 2; ++dt)
            for (int64_t t : {(int64_t)0, (int64_t)1, (int64_t)65, (int64_t)1 << 20, far})
                for (int back = 0; back < 2; ++back) {
                    kda_glu_dims_t g = {};
                    g.tokens = t; g.width = z[0]; g.hidden = z[1]; g.dtype = dt; g.activation = KDA_ACT_GELU;
                    n = 0;
                    const int got = kda_glu_workspace_size(&g, p, p, p, back, &n);
                    if (got == KDA_OK && back && n < (uint64_t)t * z[1] * (dt ? 4 : 12)) ++bad;
                    if (got == KDA_OK && n > 256)
                        expect(back ? kda_glu_bwd(&g, p, p, p, f, p, p, p, p, p, 255, nullptr)
                                    : kda_glu_fwd(&g, p, p, p, p, f, p, 255, nullptr),
                               t ? KDA_ERR_INVALID_ARGUMENT : back ? KDA_ERR_INVALID_ARGUMENT : KDA_OK, "glu small");
                }
    kda_glu_dims_t g = {};
    g.tokens = 4; g.width = 64; g.hidden = 64; g.dtype = KDA_BF16; g.activation = KDA_ACT_SILU; g.x_stride = INT64_MIN;
    expect(kda_glu_fwd(&g, p, p, p, p, nullptr, nullptr, 0, nullptr), KDA_ERR_INVALID_ARGUMENT, "glu stride");
    g.x_stride = INT64_MAX;
    kda_glu_workspace_size(&g, p, p, p, 1, &n);

    kda_state_cache_dims_t c = {};
    c.states = 0x7fffffff; c.slots = 0x7fffffff; c.rows = (int64_t)1 << 40; c.width = 8192;
    expect(kda_state_cache_write(&c, f, cu, p, f, nullptr), KDA_ERR_INVALID_ARGUMENT, "cache states");
    c.states = 1 << 20;
    expect(kda_state_cache_read(&c, p, f, cu, f, nullptr), KDA_ERR_INVALID_ARGUMENT, "cache rows");
    c.states = 0; c.slots = 0;
    expect(kda_state_cache_read(&c, p, f, cu, f, nullptr), KDA_OK, "cache empty");

    if (bad) return 1;
    printf("mixer api sanitizer check ok\n");
    return 0;
}
