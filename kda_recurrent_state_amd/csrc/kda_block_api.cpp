// kda_block_api.cpp -- the extern "C" entry points of the operators around the
// state layer (include/kda.h): argument validation, workspace layout, launch.
// Nothing here allocates device memory or keeps state.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_block.hpp"
#include "kda_checks.hpp"

using namespace kda::checks;

namespace {

// ---------------------------------------------------------------- kda_scan

int plan_scan(const kda_scan_dims_t* d, kda::LinScanArgs* a) {
    if (!d) return fail(KDA_ERR_INVALID_ARGUMENT, "dims is NULL");
    KDA_TRY(check_packed(d->num_seqs, d->total_tokens, d->channels, d->dtype, d->reserved));
    *a = kda::LinScanArgs();
    a->N = d->num_seqs;
    a->T = (int32_t)d->total_tokens;
    a->C = d->channels;
    a->dtype = d->dtype;
    KDA_TRY(check_stride(&a->xs, d->x_stride, a->C, "x_stride"));
    KDA_TRY(check_stride(&a->ls, d->log_a_stride, a->C, "log_a_stride"));
    KDA_TRY(check_stride(&a->ds, d->dy_stride, a->C, "dy_stride"));
    return KDA_OK;
}

size_t scan_chain_bytes(const kda::LinScanArgs& a) { return round256(kda::linscan_chain_bytes(a.T, a.C)); }
size_t scan_workspace(const kda::LinScanArgs& a, int backward) {
    const size_t states = ((size_t)a.T + KDA_SCAN_STATE_EVERY - 1) / KDA_SCAN_STATE_EVERY * a.C * 4;
    return scan_chain_bytes(a) + (backward ? round256(states) : 0);
}

int check_scan_size(const kda::LinScanArgs& a) {
    if (!kda::linscan_fits(a.T, a.C))
        return fail(KDA_ERR_INVALID_ARGUMENT, "total_tokens x channels = %d x %d is too large", a.T, a.C);
    return KDA_OK;
}

// ---------------------------------------------------------------- kda_conv

int plan_conv(const kda_conv_dims_t* d, kda::ConvArgs* a) {
    if (!d) return fail(KDA_ERR_INVALID_ARGUMENT, "dims is NULL");
    KDA_TRY(check_packed(d->num_seqs, d->total_tokens, d->channels, d->dtype, d->reserved));
    if (d->width < 2 || d->width > 4) return fail(KDA_ERR_UNSUPPORTED, "width = %d: must be 2, 3 or 4", d->width);
    if (d->activation != KDA_ACT_NONE && d->activation != KDA_ACT_SILU)
        return fail(KDA_ERR_INVALID_ARGUMENT, "activation = %d is not KDA_ACT_NONE or KDA_ACT_SILU", d->activation);
    *a = kda::ConvArgs();
    a->N = d->num_seqs;
    a->T = (int32_t)d->total_tokens;
    a->C = d->channels;
    a->W = d->width;
    a->dtype = d->dtype;
    a->silu = d->activation == KDA_ACT_SILU;
    KDA_TRY(check_stride(&a->xs, d->x_stride, a->C, "x_stride"));
    KDA_TRY(check_stride(&a->ds, d->dy_stride, a->C, "dy_stride"));
    return KDA_OK;
}

size_t conv_bwd_workspace(const kda::ConvArgs& a) {
    return round256((size_t)kda::conv_bwd_parts(a.T, a.N, a.C) * a.C * (a.W + 1) * 4);
}

// ---------------------------------------------------------------- norms

int check_norm(int64_t rows_max, int64_t tokens, int64_t heads, int32_t width, float eps, int32_t reserved) {
    if (tokens < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "tokens = %lld < 0", (long long)tokens);
    if (heads < 1) return fail(KDA_ERR_INVALID_ARGUMENT, "heads = %lld < 1", (long long)heads);
    if (tokens > rows_max / heads)
        return fail(KDA_ERR_INVALID_ARGUMENT, "tokens x heads = %lld x %lld: at most %lld rows", (long long)tokens,
                    (long long)heads, (long long)rows_max);
    if (width < 1) return fail(KDA_ERR_INVALID_ARGUMENT, "width = %d < 1", width);
    if (width > kMaxWidth) return fail(KDA_ERR_UNSUPPORTED, "width = %d: at most %d", width, kMaxWidth);
    if (!(eps >= 0.f) || isinf(eps)) return fail(KDA_ERR_INVALID_ARGUMENT, "eps = %g must be finite and >= 0", (double)eps);
    if (reserved != 0) return fail(KDA_ERR_INVALID_ARGUMENT, "reserved = %d is not 0", reserved);
    return KDA_OK;
}

int plan_norm_gate(const kda_norm_gate_dims_t* d, kda::NormGateArgs* a) {
    if (!d) return fail(KDA_ERR_INVALID_ARGUMENT, "dims is NULL");
    KDA_TRY(check_norm(kMaxTokens, d->tokens, d->heads, d->width, d->eps, d->reserved));
    KDA_TRY(check_dtype(d->dtype, "dtype"));
    *a = kda::NormGateArgs();
    a->rows = d->tokens * d->heads;
    a->heads = d->heads;
    a->width = d->width;
    a->eps = d->eps;
    a->dtype = d->dtype;
    a->silu = d->activation == KDA_ACT_SILU;
    const int64_t token = (int64_t)d->heads * d->width;
    KDA_TRY(check_stride(&a->xs, d->x_stride, token, "x_stride"));
    KDA_TRY(check_stride(&a->gs, d->gate_stride, token, "gate_stride"));
    KDA_TRY(check_stride(&a->ds, d->dy_stride, token, "dy_stride"));
    return KDA_OK;
}

int check_gate_act(const kda_norm_gate_dims_t* d, const void* gate) {
    if (gate && d->activation != KDA_ACT_SILU && d->activation != KDA_ACT_SIGMOID)
        return fail(KDA_ERR_INVALID_ARGUMENT, "activation = %d is not KDA_ACT_SILU or KDA_ACT_SIGMOID", d->activation);
    return KDA_OK;
}

size_t norm_gate_workspace(const kda::NormGateArgs& a) {
    return round256((size_t)kda::norm_gate_blocks(a.dtype, a.width, a.rows) * a.width * 4);
}

int plan_res_norm(const kda_residual_norm_dims_t* d, kda::ResNormArgs* a) {
    if (!d) return fail(KDA_ERR_INVALID_ARGUMENT, "dims is NULL");
    KDA_TRY(check_norm(kMaxTokens, d->tokens, 1, d->width, d->eps, d->reserved));
    KDA_TRY(check_dtype(d->dtype, "dtype"));
    KDA_TRY(check_dtype(d->residual_dtype, "residual_dtype"));
    if (d->dtype == KDA_F32 && d->residual_dtype == KDA_BF16)
        return fail(KDA_ERR_UNSUPPORTED, "a bf16 residual with float32 inputs is not compiled");
    if (!isfinite(d->scale)) return fail(KDA_ERR_INVALID_ARGUMENT, "scale = %g is not finite", (double)d->scale);
    *a = kda::ResNormArgs();
    a->rows = d->tokens;
    a->width = d->width;
    a->eps = d->eps;
    a->scale = d->scale;
    a->dtype = d->dtype;
    a->rdtype = d->residual_dtype;
    KDA_TRY(check_stride(&a->xs, d->x_stride, d->width, "x_stride"));
    KDA_TRY(check_stride(&a->rs, d->residual_stride, d->width, "residual_stride"));
    KDA_TRY(check_stride(&a->ds, d->dy_stride, d->width, "dy_stride"));
    KDA_TRY(check_stride(&a->drs, d->dresidual_stride, d->width, "dresidual_stride"));
    return KDA_OK;
}

// the larger of the backward's two layouts (with and without dchannel_scale)
size_t res_norm_workspace(kda::ResNormArgs a) {
    size_t most = 0;
    for (int dcs = 0; dcs < 2; ++dcs) {
        a.want_dcs = dcs;
        const size_t bytes = (size_t)kda::res_norm_blocks(a) * a.width * (dcs + 1) * 4;
        if (bytes > most) most = bytes;
    }
    return round256(most);
}

}  // namespace

extern "C" {

int kda_scan_workspace_size(const kda_scan_dims_t* d, int backward, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    kda::LinScanArgs a;
    KDA_TRY(plan_scan(d, &a));
    *bytes = scan_workspace(a, backward);
    return ok();
}

int kda_scan_fwd(const kda_scan_dims_t* d, const void* x, const float* log_a, const float* h0, const int32_t* cu_seqlens,
                 void* y, float* h_T, float* states, void* workspace, size_t workspace_bytes, void* stream) {
    kda::LinScanArgs a;
    KDA_TRY(plan_scan(d, &a));
    KDA_TRY(check_lengths(a.N, a.T, cu_seqlens));
    if (a.N == 0) return ok();
    const int e = esize(a.dtype);
    if (a.T > 0) {
        const void* ptrs[] = {x, log_a, y};
        const char* names[] = {"x", "log_a", "y"};
        const int align[] = {e, 4, e};
        KDA_TRY(check_ptrs(ptrs, names, align, 3));
    }
    KDA_TRY(check_optional(h0, 4, "h0"));
    KDA_TRY(check_optional(h_T, 4, "h_T"));
    KDA_TRY(check_optional(states, 4, "states"));
    if (h_T && h_T == h0) return fail(KDA_ERR_INVALID_ARGUMENT, "h_T must not be h0");
    KDA_TRY(check_workspace(workspace, workspace_bytes, scan_workspace(a, 0)));
    KDA_TRY(check_scan_size(a));
    a.x = x; a.la = log_a; a.h0 = h0; a.cu = cu_seqlens; a.eq = cu_seqlens ? 0 : a.T / a.N;
    a.y = y; a.hT = h_T; a.states = states;
    a.word = static_cast<uint64_t*>(workspace);
    return hip_status(kda::launch_linscan_fwd(a, true, (hipStream_t)stream), "scan");
}

int kda_scan_bwd(const kda_scan_dims_t* d, const void* x, const float* log_a, const float* h0, const int32_t* cu_seqlens,
                 const float* states, const void* dy, const float* dh_T, void* dx, float* dlog_a, float* dh0,
                 void* workspace, size_t workspace_bytes, void* stream) {
    kda::LinScanArgs a;
    KDA_TRY(plan_scan(d, &a));
    KDA_TRY(check_lengths(a.N, a.T, cu_seqlens));
    if (a.N == 0) return ok();
    const int e = esize(a.dtype);
    if (a.T > 0) {
        const void* ptrs[] = {x, log_a, dy, dx, dlog_a};
        const char* names[] = {"x", "log_a", "dy", "dx", "dlog_a"};
        const int align[] = {e, 4, e, e, 4};
        KDA_TRY(check_ptrs(ptrs, names, align, 5));
    }
    KDA_TRY(check_optional(h0, 4, "h0"));
    KDA_TRY(check_optional(states, 4, "states"));
    KDA_TRY(check_optional(dh_T, 4, "dh_T"));
    KDA_TRY(check_optional(dh0, 4, "dh0"));
    if (dh0 && (dh0 == dh_T || dh0 == h0)) return fail(KDA_ERR_INVALID_ARGUMENT, "dh0 must not be dh_T or h0");
    KDA_TRY(check_workspace(workspace, workspace_bytes, scan_workspace(a, 1)));
    KDA_TRY(check_scan_size(a));
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.x = x; a.la = log_a; a.h0 = h0; a.cu = cu_seqlens; a.eq = cu_seqlens ? 0 : a.T / a.N;
    a.dy = dy; a.dhT = dh_T; a.y = dx; a.dla = dlog_a; a.hT = dh0;
    a.word = reinterpret_cast<uint64_t*>(ws);
    if (states) {
        a.states = const_cast<float*>(states);
    } else {
        a.states = reinterpret_cast<float*>(ws + scan_chain_bytes(a));
        KDA_TRY(hip_status(kda::launch_linscan_fwd(a, false, (hipStream_t)stream), "scan"));
    }
    return hip_status(kda::launch_linscan_bwd(a, (hipStream_t)stream), "scan gradient");
}

int kda_scan_step(const kda_scan_dims_t* d, const void* x, const float* log_a, const float* h_in, float* h_out, void* y,
                  void* stream) {
    kda::LinScanArgs a;
    KDA_TRY(plan_scan(d, &a));
    if (a.T != a.N)
        return fail(KDA_ERR_INVALID_ARGUMENT, "a step needs total_tokens (%d) == num_seqs (%d)", a.T, a.N);
    if (a.N == 0) return ok();
    const int e = esize(a.dtype);
    const void* ptrs[] = {x, log_a, h_in, h_out, y};
    const char* names[] = {"x", "log_a", "h_in", "h_out", "y"};
    const int align[] = {e, 4, 4, 4, e};
    KDA_TRY(check_ptrs(ptrs, names, align, 5));
    if ((int64_t)a.N * a.C > kMaxThreads) return fail(KDA_ERR_INVALID_ARGUMENT, "too many states: %d x %d", a.N, a.C);
    a.x = x; a.la = log_a; a.h0 = h_in; a.hT = h_out; a.y = y;
    return hip_status(kda::launch_linscan_step(a, (hipStream_t)stream), "scan step");
}

int kda_conv_fwd(const kda_conv_dims_t* d, const void* x, const float* weight, const float* bias, const void* state,
                 const int32_t* cu_seqlens, void* y, void* state_T, void* stream) {
    kda::ConvArgs a;
    KDA_TRY(plan_conv(d, &a));
    KDA_TRY(check_lengths(a.N, a.T, cu_seqlens));
    if (a.N == 0) return ok();
    const int e = esize(a.dtype);
    const void* ptrs[] = {weight, x, y};
    const char* names[] = {"weight", "x", "y"};
    const int align[] = {4, e, e};
    KDA_TRY(check_ptrs(ptrs, names, align, a.T > 0 ? 3 : 1));
    KDA_TRY(check_optional(bias, 4, "bias"));
    KDA_TRY(check_optional(state, e, "state"));
    KDA_TRY(check_optional(state_T, e, "state_T"));
    if (state_T && state_T == state) return fail(KDA_ERR_INVALID_ARGUMENT, "state_T must not be state");
    a.x = x; a.weight = weight; a.bias = bias; a.state = state; a.cu = cu_seqlens; a.eq = cu_seqlens ? 0 : a.T / a.N;
    a.y = y; a.state_T = state_T;
    return hip_status(kda::launch_conv_fwd(a, (hipStream_t)stream), "convolution");
}

int kda_conv_bwd_workspace_size(const kda_conv_dims_t* d, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    kda::ConvArgs a;
    KDA_TRY(plan_conv(d, &a));
    *bytes = conv_bwd_workspace(a);
    return ok();
}

int kda_conv_bwd(const kda_conv_dims_t* d, const void* x, const float* weight, const float* bias, const void* state,
                 const int32_t* cu_seqlens, const void* dy, const void* dstate_T, void* dx, float* dweight, float* dbias,
                 void* dstate, void* workspace, size_t workspace_bytes, void* stream) {
    kda::ConvArgs a;
    KDA_TRY(plan_conv(d, &a));
    KDA_TRY(check_lengths(a.N, a.T, cu_seqlens));
    const int e = esize(a.dtype);
    const void* ptrs[] = {weight, x, dy, dx};
    const char* names[] = {"weight", "x", "dy", "dx"};
    const int align[] = {4, e, e, e};
    KDA_TRY(check_ptrs(ptrs, names, align, a.T > 0 ? 4 : 1));
    KDA_TRY(check_optional(bias, 4, "bias"));
    KDA_TRY(check_optional(state, e, "state"));
    KDA_TRY(check_optional(dstate_T, e, "dstate_T"));
    KDA_TRY(check_optional(dweight, 4, "dweight"));
    KDA_TRY(check_optional(dbias, 4, "dbias"));
    KDA_TRY(check_optional(dstate, e, "dstate"));
    if (dstate && (dstate == state || dstate == dstate_T))
        return fail(KDA_ERR_INVALID_ARGUMENT, "dstate must not be state or dstate_T");
    KDA_TRY(check_workspace(workspace, workspace_bytes, conv_bwd_workspace(a)));
    a.x = x; a.weight = weight; a.bias = bias; a.state = state;
    a.cu = cu_seqlens; a.eq = cu_seqlens || a.N == 0 ? 0 : a.T / a.N;
    a.dy = dy; a.dstT = dstate_T; a.y = dx; a.state_T = dstate;
    a.part = static_cast<float*>(workspace);
    if (a.N > 0) KDA_TRY(hip_status(kda::launch_conv_bwd(a, (hipStream_t)stream), "convolution gradient"));
    if (!dweight && !dbias) return ok();
    return hip_status(kda::launch_colsum(a.part, kda::conv_bwd_parts(a.T, a.N, a.C), (int64_t)a.C * (a.W + 1),
                                         (int64_t)a.C * a.W, dweight, dbias, (hipStream_t)stream),
                      "convolution gradient");
}

int kda_conv_step(const kda_conv_dims_t* d, const void* x, const float* weight, const float* bias, const void* state_in,
                  void* state_out, void* y, void* stream) {
    kda::ConvArgs a;
    KDA_TRY(plan_conv(d, &a));
    if (a.T != a.N)
        return fail(KDA_ERR_INVALID_ARGUMENT, "a step needs total_tokens (%d) == num_seqs (%d)", a.T, a.N);
    if (a.N == 0) return ok();
    const int e = esize(a.dtype);
    const void* ptrs[] = {x, weight, state_in, state_out, y};
    const char* names[] = {"x", "weight", "state_in", "state_out", "y"};
    const int align[] = {e, 4, e, e, e};
    KDA_TRY(check_ptrs(ptrs, names, align, 5));
    KDA_TRY(check_optional(bias, 4, "bias"));
    if ((int64_t)a.N * a.C > kMaxThreads) return fail(KDA_ERR_INVALID_ARGUMENT, "too many states: %d x %d", a.N, a.C);
    a.x = x; a.weight = weight; a.bias = bias; a.state = state_in; a.state_T = state_out; a.y = y;
    return hip_status(kda::launch_conv_step(a, (hipStream_t)stream), "convolution step");
}

int kda_norm_gate_fwd(const kda_norm_gate_dims_t* d, const void* x, const float* weight, const void* gate, void* y,
                      void* stream) {
    kda::NormGateArgs a;
    KDA_TRY(plan_norm_gate(d, &a));
    KDA_TRY(check_gate_act(d, gate));
    if (a.rows == 0) return ok();
    const int e = esize(a.dtype);
    const void* ptrs[] = {x, y};
    const char* names[] = {"x", "y"};
    const int align[] = {e, e};
    KDA_TRY(check_ptrs(ptrs, names, align, 2));
    KDA_TRY(check_optional(weight, 4, "weight"));
    KDA_TRY(check_optional(gate, e, "gate"));
    if (y == x && a.xs != (int64_t)d->heads * d->width)
        return fail(KDA_ERR_INVALID_ARGUMENT, "y may be x only where x is contiguous");
    a.x = x; a.weight = weight; a.gate = gate; a.y = y;
    return hip_status(kda::launch_norm_gate(a, false, (hipStream_t)stream), "norm");
}

int kda_norm_gate_bwd_workspace_size(const kda_norm_gate_dims_t* d, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    kda::NormGateArgs a;
    KDA_TRY(plan_norm_gate(d, &a));
    *bytes = norm_gate_workspace(a);
    return ok();
}

int kda_norm_gate_bwd(const kda_norm_gate_dims_t* d, const void* x, const float* weight, const void* gate,
                      const void* dy, void* dx, void* dgate, float* dweight, void* workspace, size_t workspace_bytes,
                      void* stream) {
    kda::NormGateArgs a;
    KDA_TRY(plan_norm_gate(d, &a));
    KDA_TRY(check_gate_act(d, gate));
    const int e = esize(a.dtype);
    if (a.rows > 0) {
        const void* ptrs[] = {x, dy, dx};
        const char* names[] = {"x", "dy", "dx"};
        const int align[] = {e, e, e};
        KDA_TRY(check_ptrs(ptrs, names, align, 3));
        if (!gate != !dgate) return fail(KDA_ERR_INVALID_ARGUMENT, "gate and dgate go together");
    }
    KDA_TRY(check_optional(weight, 4, "weight"));
    KDA_TRY(check_optional(gate, e, "gate"));
    KDA_TRY(check_optional(dgate, e, "dgate"));
    KDA_TRY(check_optional(dweight, 4, "dweight"));
    if (dweight) KDA_TRY(check_workspace(workspace, workspace_bytes, norm_gate_workspace(a)));
    a.x = x; a.weight = weight; a.gate = gate; a.dy = dy; a.y = dx; a.dgate = dgate;
    a.part = dweight ? static_cast<float*>(workspace) : nullptr;
    if (a.rows > 0) KDA_TRY(hip_status(kda::launch_norm_gate(a, true, (hipStream_t)stream), "norm gradient"));
    if (!dweight) return ok();
    return hip_status(kda::launch_colsum(a.part, kda::norm_gate_blocks(a.dtype, a.width, a.rows), a.width, a.width,
                                         dweight, nullptr, (hipStream_t)stream),
                      "norm gradient");
}

int kda_residual_norm_fwd(const kda_residual_norm_dims_t* d, const void* x, const void* residual, const float* weight,
                          const float* channel_scale, void* residual_out, void* y, void* stream) {
    kda::ResNormArgs a;
    KDA_TRY(plan_res_norm(d, &a));
    if (a.rows == 0) return ok();
    const int e = esize(a.dtype), er = esize(a.rdtype);
    const void* ptrs[] = {x, residual, weight, residual_out, y};
    const char* names[] = {"x", "residual", "weight", "residual_out", "y"};
    const int align[] = {e, er, 4, er, e};
    KDA_TRY(check_ptrs(ptrs, names, align, 5));
    KDA_TRY(check_optional(channel_scale, 4, "channel_scale"));
    if (residual_out == residual && a.rs != a.width)
        return fail(KDA_ERR_INVALID_ARGUMENT, "residual_out may be residual only where residual is contiguous");
    a.x = x; a.res = residual; a.weight = weight; a.cscale = channel_scale; a.res_out = residual_out; a.y = y;
    return hip_status(kda::launch_res_norm(a, false, (hipStream_t)stream), "residual norm");
}

int kda_residual_norm_bwd_workspace_size(const kda_residual_norm_dims_t* d, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    kda::ResNormArgs a;
    KDA_TRY(plan_res_norm(d, &a));
    *bytes = res_norm_workspace(a);
    return ok();
}

int kda_residual_norm_bwd(const kda_residual_norm_dims_t* d, const void* x, const void* residual_out,
                          const float* weight, const float* channel_scale, const void* dy, const void* dresidual_out,
                          void* dx, void* dresidual, float* dweight, float* dchannel_scale, void* workspace,
                          size_t workspace_bytes, void* stream) {
    kda::ResNormArgs a;
    KDA_TRY(plan_res_norm(d, &a));
    const int e = esize(a.dtype), er = esize(a.rdtype);
    if (a.rows > 0) {
        const void* ptrs[] = {residual_out, weight, dy, dx, dresidual, x};
        const char* names[] = {"residual_out", "weight", "dy", "dx", "dresidual", "x"};
        const int align[] = {er, 4, e, e, er, e};
        KDA_TRY(check_ptrs(ptrs, names, align, dchannel_scale ? 6 : 5));
    }
    KDA_TRY(check_optional(channel_scale, 4, "channel_scale"));
    KDA_TRY(check_optional(dresidual_out, er, "dresidual_out"));
    KDA_TRY(check_optional(dweight, 4, "dweight"));
    KDA_TRY(check_optional(dchannel_scale, 4, "dchannel_scale"));
    const bool sums = dweight || dchannel_scale;
    if (sums) KDA_TRY(check_workspace(workspace, workspace_bytes, res_norm_workspace(a)));
    a.x = x; a.res = residual_out; a.weight = weight; a.cscale = channel_scale; a.dy = dy; a.dres = dresidual_out;
    a.res_out = dresidual; a.y = dx;
    a.part = sums ? static_cast<float*>(workspace) : nullptr;
    a.want_dcs = dchannel_scale != nullptr;
    if (a.rows > 0) KDA_TRY(hip_status(kda::launch_res_norm(a, true, (hipStream_t)stream), "residual norm gradient"));
    if (!sums) return ok();
    return hip_status(kda::launch_colsum(a.part, kda::res_norm_blocks(a),
                                         (int64_t)a.width * (a.want_dcs ? 2 : 1), a.width, dweight, dchannel_scale,
                                         (hipStream_t)stream),
                      "residual norm gradient");
}

}  // extern "C"
