// kda_ssm_api.cpp -- the extern "C" entry points of the selective state space scan
// (include/kda.h): argument validation, plan, workspace layout, launch.  Nothing
// here allocates device memory or keeps state.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_checks.hpp"
#include "kda_ssm.hpp"

using namespace kda::checks;

namespace {

constexpr int kMaxHeads = 65536;
constexpr int kMaxHeadWidth = 8192;
constexpr int64_t kMaxBlocks = 0xffffff;  // workgroups of 256 threads in one launch
constexpr int64_t kWalkGroups = 768;
constexpr int kWaves = 4;                 // units of a workgroup of the walk

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

int check_dims(const kda_ssm_dims_t* d) {
    if (!d) return fail(KDA_ERR_INVALID_ARGUMENT, "dims is NULL");
    KDA_TRY(check_packed(d->num_seqs, d->total_tokens, 1, d->dtype, d->reserved));
    if (d->heads < 1 || d->heads > kMaxHeads)
        return fail(KDA_ERR_INVALID_ARGUMENT, "heads = %d: must be 1 to %d", d->heads, kMaxHeads);
    if (d->groups < 1 || d->heads % d->groups)
        return fail(KDA_ERR_INVALID_ARGUMENT, "groups = %d: must divide heads = %d", d->groups, d->heads);
    if (d->width < 1) return fail(KDA_ERR_INVALID_ARGUMENT, "width = %d < 1", d->width);
    if (d->width > kMaxHeadWidth) return fail(KDA_ERR_UNSUPPORTED, "width = %d: at most %d", d->width, kMaxHeadWidth);
    if (d->state < 1) return fail(KDA_ERR_INVALID_ARGUMENT, "state = %d < 1", d->state);
    if (d->state > kda::SSM_MAX_STATE)
        return fail(KDA_ERR_UNSUPPORTED, "state = %d: at most %d", d->state, kda::SSM_MAX_STATE);
    if (d->softplus != 0 && d->softplus != 1)
        return fail(KDA_ERR_INVALID_ARGUMENT, "softplus = %d is not 0 or 1", d->softplus);
    return KDA_OK;
}

int plan(const kda_ssm_dims_t* d, kda::SsmArgs* a) {
    KDA_TRY(check_dims(d));
    *a = kda::SsmArgs();
    a->N = d->num_seqs;
    a->T = (int32_t)d->total_tokens;
    a->H = d->heads;
    a->G = d->groups;
    a->K = d->state;
    a->P = d->width;
    a->dtype = d->dtype;
    a->softplus = d->softplus;
    KDA_TRY(check_stride(&a->xs, d->x_stride, (int64_t)a->H * a->P, "x_stride"));
    KDA_TRY(check_stride(&a->dts, d->dt_stride, a->H, "dt_stride"));
    KDA_TRY(check_stride(&a->bs, d->b_stride, (int64_t)a->G * a->K, "b_stride"));
    KDA_TRY(check_stride(&a->cs, d->c_stride, (int64_t)a->G * a->K, "c_stride"));
    KDA_TRY(check_stride(&a->dys, d->dy_stride, (int64_t)a->H * a->P, "dy_stride"));
    a->chunk = kda::ssm_chunk(a->dtype);
    a->rows = kda::ssm_rows(a->K);
    a->cols = kda::ssm_cols(a->K);
    a->blocks = (a->P + a->cols - 1) / a->cols;
    a->wcols = a->cols / 2;
    a->wblocks = (a->P + a->wcols - 1) / a->wcols;
    // Segments: enough workgroups for three on every compute unit, all that fit, so that they run in one round.  Measured
    // with workgroups for 512, 768, 1024 and 1536, us: 2 x 32768 tokens of 32 heads 920, 786, 897, 823; gradient of
    // 2 x 8192 1049, 999, 1079, 1060; 16384 tokens of 32 heads of 64 119, 115, 111, 127; one of 4096 65 each.
    const int64_t quads = ((int64_t)a->H / a->G * a->wblocks + kWaves - 1) / kWaves;
    const int64_t want = kWalkGroups / (quads * a->G) > 0 ? kWalkGroups / (quads * a->G) : 1;
    const int64_t seg = round_up((a->T + want - 1) / want, a->chunk);
    a->seg = (int32_t)(seg < 2 * a->chunk ? 2 * a->chunk : seg);
    const int64_t pairs = kda::ssm_slots(*a, a->chunk) * a->G, units = (int64_t)a->H / a->G * a->blocks;
    const int64_t split = pairs > 0 ? (512 + pairs - 1) / pairs : 1;
    a->split = (int32_t)(split < units ? split : units);
    return KDA_OK;
}

// The workspace's arrays, in order; returns its size.
size_t layout(kda::SsmArgs* a, int backward, uint8_t* base) {
    size_t at = 0;
    auto take = [&](int64_t floats) {
        float* p = base ? reinterpret_cast<float*>(base + at) : nullptr;
        at += round256((size_t)floats * 4);
        return p;
    };
    const int64_t units = kda::ssm_units(*a);
    if (a->seg < a->T) {
        const int64_t slots = kda::ssm_slots(*a, a->seg);
        a->ends = take(slots * a->H * a->wblocks * a->rows * a->wcols);
        a->decay = take(slots * a->H);
        if (backward) {
            a->rends = take(slots * a->H * a->wblocks * a->rows * a->wcols);
            a->rdecay = take(slots * a->H);
        }
    }
    if (backward) {
        const int64_t slots = kda::ssm_slots(*a, a->chunk);
        a->hs = take(slots * units * kda::ssm_unit_state(*a));
        a->gs = take(slots * units * kda::ssm_unit_state(*a));
        if (a->split > 1) a->part = take((int64_t)a->split * 2 * a->T * a->G * a->K);
        a->dec = take(slots * a->H * kda::ssm_decay_floats(*a));
        a->tok = take(slots * units * kda::ssm_token_floats(a->chunk));
        a->sums = take(slots * 3 * a->H);
    }
    return at;
}

// A launch holds 2^32 threads, and the states of a gradient's chunks less than 2^60 bytes.  In double, which holds every
// product of the sizes' limits.
int check_size(const kda::SsmArgs& a, int backward) {
    const double quads = ((int64_t)a.H / a.G * a.wblocks + kWaves - 1) / kWaves, chunks = kda::ssm_slots(a, a.chunk);
    const double walk = ((double)kda::ssm_slots(a, a.seg) * a.G + 8) * quads * (backward ? 2 : 1);
    const double grad = backward ? fmax((chunks * a.G + 8) * a.split, chunks * a.H / 4 + 1) : 0;
    const double states = backward ? chunks * a.H * a.blocks * a.rows * a.cols * 8 : 0;
    if (walk > kMaxBlocks || grad > kMaxBlocks || states > 1e18)
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs, total_tokens and heads = %d, %d and %d are too large for one launch",
                    a.N, a.T, a.H);
    return KDA_OK;
}

int check_inputs(const kda::SsmArgs& a, const void* x, const float* dt, const float* A, const void* B, const void* C,
                 const float* D, const float* dt_bias, const float* h0) {
    const int e = esize(a.dtype);
    const void* ptrs[] = {A, x, dt, B, C};
    const char* names[] = {"A", "x", "dt", "B", "C"};
    const int align[] = {4, e, 4, e, e};
    KDA_TRY(check_ptrs(ptrs, names, align, a.T > 0 ? 5 : 1));
    KDA_TRY(check_optional(D, 4, "D"));
    KDA_TRY(check_optional(dt_bias, 4, "dt_bias"));
    return check_optional(h0, 4, "h0");
}

}  // namespace

extern "C" {

int kda_ssm_workspace_size(const kda_ssm_dims_t* d, int backward, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    kda::SsmArgs a;
    KDA_TRY(plan(d, &a));
    KDA_TRY(check_size(a, backward));
    *bytes = layout(&a, backward, nullptr);
    return ok();
}

int kda_ssm_fwd(const kda_ssm_dims_t* d, const void* x, const float* dt, const float* A, const void* B, const void* C,
                const float* D, const float* dt_bias, const float* h0, const int32_t* cu_seqlens, void* y, float* h_T,
                void* workspace, size_t workspace_bytes, void* stream) {
    kda::SsmArgs a;
    KDA_TRY(plan(d, &a));
    KDA_TRY(check_lengths(a.N, a.T, cu_seqlens));
    if (a.N == 0) return ok();
    KDA_TRY(check_inputs(a, x, dt, A, B, C, D, dt_bias, h0));
    if (a.T > 0 && !y) return fail(KDA_ERR_INVALID_ARGUMENT, "y is NULL");
    KDA_TRY(check_optional(y, esize(a.dtype), "y"));
    KDA_TRY(check_optional(h_T, 4, "h_T"));
    if (h_T && h_T == h0) return fail(KDA_ERR_INVALID_ARGUMENT, "h_T must not be h0");
    KDA_TRY(check_size(a, 0));
    KDA_TRY(check_workspace(workspace, workspace_bytes, layout(&a, 0, nullptr)));
    layout(&a, 0, static_cast<uint8_t*>(workspace));
    a.x = x; a.dt = dt; a.A = A; a.B = B; a.C = C; a.D = D; a.bias = dt_bias; a.h0 = h0;
    a.cu = cu_seqlens; a.eq = cu_seqlens ? 0 : a.T / a.N;
    a.y = y; a.hT = h_T;
    return hip_status(kda::launch_ssm_fwd(a, (hipStream_t)stream), "state space scan");
}

int kda_ssm_bwd(const kda_ssm_dims_t* d, const void* x, const float* dt, const float* A, const void* B, const void* C,
                const float* D, const float* dt_bias, const float* h0, const int32_t* cu_seqlens, const void* dy,
                const float* dh_T, void* dx, float* ddt, float* dA, void* dB, void* dC, float* dD, float* ddt_bias,
                float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
    kda::SsmArgs a;
    KDA_TRY(plan(d, &a));
    KDA_TRY(check_lengths(a.N, a.T, cu_seqlens));
    KDA_TRY(check_inputs(a, x, dt, A, B, C, D, dt_bias, h0));
    const int e = esize(a.dtype);
    if (a.T > 0) {
        const void* ptrs[] = {dy, dx, ddt, dB, dC};
        const char* names[] = {"dy", "dx", "ddt", "dB", "dC"};
        const int align[] = {e, e, 4, e, e};
        KDA_TRY(check_ptrs(ptrs, names, align, 5));
    }
    KDA_TRY(check_optional(dh_T, 4, "dh_T"));
    KDA_TRY(check_optional(dA, 4, "dA"));
    KDA_TRY(check_optional(dD, 4, "dD"));
    KDA_TRY(check_optional(ddt_bias, 4, "ddt_bias"));
    KDA_TRY(check_optional(dh0, 4, "dh0"));
    if (dh0 && (dh0 == dh_T || dh0 == h0)) return fail(KDA_ERR_INVALID_ARGUMENT, "dh0 must not be dh_T or h0");
    KDA_TRY(check_size(a, 1));
    KDA_TRY(check_workspace(workspace, workspace_bytes, layout(&a, 1, nullptr)));
    layout(&a, 1, static_cast<uint8_t*>(workspace));
    a.x = x; a.dt = dt; a.A = A; a.B = B; a.C = C; a.D = D; a.bias = dt_bias; a.h0 = h0;
    a.cu = cu_seqlens; a.eq = cu_seqlens || a.N == 0 ? 0 : a.T / a.N;
    a.dy = dy; a.dhT = dh_T; a.y = dx; a.ddt = ddt; a.dA = dA; a.dB = dB; a.dC = dC; a.dD = dD; a.dbias = ddt_bias;
    a.dh0 = dh0;
    return hip_status(kda::launch_ssm_bwd(a, (hipStream_t)stream), "state space scan gradient");
}

namespace {

int check_step(const kda_ssm_dims_t* d, const float* dt, const float* A, const float* D, const float* dt_bias,
               const float* h_in, float* h_out, void* y) {
    KDA_TRY(check_dims(d));
    if (d->total_tokens != d->num_seqs)
        return fail(KDA_ERR_INVALID_ARGUMENT, "a step needs total_tokens (%lld) == num_seqs (%d)",
                    (long long)d->total_tokens, d->num_seqs);
    const void* ptrs[] = {dt, A, h_in, h_out, y};
    const char* names[] = {"dt", "A", "h_in", "h_out", "y"};
    const int align[] = {4, 4, 4, 4, esize(d->dtype)};
    KDA_TRY(check_ptrs(ptrs, names, align, d->num_seqs ? 5 : 0));
    KDA_TRY(check_optional(D, 4, "D"));
    KDA_TRY(check_optional(dt_bias, 4, "dt_bias"));
    // 8 lanes of a column each is the narrowest block of columns
    if ((int64_t)d->num_seqs * d->heads > kMaxBlocks / ((d->width + 7) / 8))
        return fail(KDA_ERR_INVALID_ARGUMENT, "too many states: %d x %d", d->num_seqs, d->heads);
    return KDA_OK;
}

kda::SsmStepArgs step_args(const kda_ssm_dims_t* d, const float* dt, const float* A, const float* D, const float* dt_bias,
                           const float* h_in, float* h_out, void* y) {
    kda::SsmStepArgs a = {};
    a.dt = dt; a.A = A; a.D = D; a.bias = dt_bias; a.h_in = h_in; a.h_out = h_out; a.y = y;
    a.N = d->num_seqs; a.H = d->heads; a.G = d->groups; a.K = d->state; a.P = d->width;
    a.dtype = d->dtype; a.softplus = d->softplus;
    return a;
}

int64_t state_bytes(const kda::SsmStepArgs& a) { return (int64_t)a.N * a.H * a.K * a.P * 4; }
Extent dt_extent(const kda::SsmStepArgs& a) { return {"dt", a.dt, a.N, a.dts * 4, 4ll * a.H}; }
Extent y_extent(const kda::SsmStepArgs& a) { return whole("y", a.y, (int64_t)a.N * a.H * a.P * esize(a.dtype)); }
// A state may be updated in place.
Extent h_in_extent(const kda::SsmStepArgs& a) { return whole("h_in", a.h_in == a.h_out ? nullptr : a.h_in, state_bytes(a)); }

}  // namespace

int kda_ssm_step(const kda_ssm_dims_t* d, const void* x, const float* dt, const float* A, const void* B, const void* C,
                 const float* D, const float* dt_bias, const float* h_in, float* h_out, void* y, void* stream) {
    KDA_TRY(check_step(d, dt, A, D, dt_bias, h_in, h_out, y));
    kda::SsmStepArgs a = step_args(d, dt, A, D, dt_bias, h_in, h_out, y);
    KDA_TRY(check_stride(&a.xs, d->x_stride, (int64_t)a.H * a.P, "x_stride"));
    KDA_TRY(check_stride(&a.dts, d->dt_stride, a.H, "dt_stride"));
    KDA_TRY(check_stride(&a.bs, d->b_stride, (int64_t)a.G * a.K, "b_stride"));
    KDA_TRY(check_stride(&a.cs, d->c_stride, (int64_t)a.G * a.K, "c_stride"));
    if (a.N == 0) return ok();
    const int e = esize(a.dtype);
    const void* ptrs[] = {x, B, C};
    const char* names[] = {"x", "B", "C"};
    const int align[] = {e, e, e};
    KDA_TRY(check_ptrs(ptrs, names, align, 3));
    const int64_t state = state_bytes(a), gk = (int64_t)a.G * a.K * e;
    const Extent others[] = {{"x", x, a.N, a.xs * e, (int64_t)a.H * a.P * e}, {"B", B, a.N, a.bs * e, gk},
                             {"C", C, a.N, a.cs * e, gk}, dt_extent(a), whole("A", A, 4ll * a.H), whole("D", D, 4ll * a.H),
                             whole("dt_bias", dt_bias, 4ll * a.H), y_extent(a), h_in_extent(a)};
    KDA_TRY(check_apart("h_out", h_out, state, others, 9));
    a.x = x; a.B = B; a.C = C;
    return hip_status(kda::launch_ssm_step(a, (hipStream_t)stream), "state space step");
}

int kda_ssm_conv_step_workspace_size(const kda_ssm_dims_t* d, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    KDA_TRY(check_dims(d));
    *bytes = round256((size_t)d->num_seqs * ((size_t)d->heads * d->width + 2 * (size_t)d->groups * d->state) * 4);
    return ok();
}

int kda_ssm_conv_step(const kda_ssm_dims_t* d, int conv_width, int conv_activation, const void* xbc,
                      const float* conv_weight, const float* conv_bias, const void* conv_state_in, void* conv_state_out,
                      const float* dt, const float* A, const float* D, const float* dt_bias, const float* h_in,
                      float* h_out, void* y, void* workspace, size_t workspace_bytes, void* stream) {
    KDA_TRY(check_step(d, dt, A, D, dt_bias, h_in, h_out, y));
    if (conv_width < 2 || conv_width > 4)
        return fail(KDA_ERR_UNSUPPORTED, "conv_width = %d: must be 2, 3 or 4", conv_width);
    if (conv_activation != KDA_ACT_NONE && conv_activation != KDA_ACT_SILU)
        return fail(KDA_ERR_INVALID_ARGUMENT, "conv_activation = %d is not KDA_ACT_NONE or KDA_ACT_SILU", conv_activation);
    kda::SsmStepArgs a = step_args(d, dt, A, D, dt_bias, h_in, h_out, y);
    const int64_t hp = (int64_t)a.H * a.P, gk = (int64_t)a.G * a.K, channels = hp + 2 * gk;
    if (channels > 1 << 24 || (int64_t)a.N * channels > kMaxBlocks * 256)
        return fail(KDA_ERR_INVALID_ARGUMENT, "too many channels: %d x %lld", a.N, (long long)channels);
    kda::SsmConvArgs c = {};
    KDA_TRY(check_stride(&c.xs, d->x_stride, channels, "x_stride"));
    KDA_TRY(check_stride(&a.dts, d->dt_stride, a.H, "dt_stride"));
    if (a.N == 0) return ok();
    const int e = esize(a.dtype);
    const void* ptrs[] = {xbc, conv_weight, conv_state_in, conv_state_out};
    const char* names[] = {"xbc", "conv_weight", "conv_state_in", "conv_state_out"};
    const int align[] = {e, 4, e, e};
    KDA_TRY(check_ptrs(ptrs, names, align, 4));
    KDA_TRY(check_optional(conv_bias, 4, "conv_bias"));
    size_t need = 0;
    kda_ssm_conv_step_workspace_size(d, &need);
    KDA_TRY(check_workspace(workspace, workspace_bytes, need));
    const int64_t state = state_bytes(a), taps = (int64_t)a.N * (conv_width - 1) * channels * e;
    const Extent others[] = {{"xbc", xbc, a.N, c.xs * e, channels * e}, whole("conv_weight", conv_weight, channels * conv_width * 4),
                             whole("conv_bias", conv_bias, channels * 4), dt_extent(a), whole("A", A, 4ll * a.H),
                             whole("D", D, 4ll * a.H), whole("dt_bias", dt_bias, 4ll * a.H), y_extent(a),
                             whole("the workspace", workspace, (int64_t)need), h_in_extent(a),
                             whole("conv_state_in", conv_state_in == conv_state_out ? nullptr : conv_state_in, taps)};
    KDA_TRY(check_apart("h_out", h_out, state, others, 11));
    KDA_TRY(check_apart("conv_state_out", conv_state_out, taps, others, 11));
    const Extent states[] = {whole("h_out", h_out, state)};
    KDA_TRY(check_apart("conv_state_out", conv_state_out, taps, states, 1));
    float* z = static_cast<float*>(workspace);
    c.x = xbc; c.weight = conv_weight; c.bias = conv_bias; c.state_in = conv_state_in; c.state_out = conv_state_out;
    c.z = z; c.N = a.N; c.C = (int32_t)channels; c.W = conv_width; c.dtype = a.dtype;
    c.silu = conv_activation == KDA_ACT_SILU;
    KDA_TRY(hip_status(kda::launch_ssm_conv(c, (hipStream_t)stream), "convolution step"));
    a.x = z; a.B = z + hp; a.C = z + hp + gk;
    a.xs = a.bs = a.cs = channels;
    a.f32_in = 1;
    return hip_status(kda::launch_ssm_step(a, (hipStream_t)stream), "state space step");
}

}  // extern "C"
