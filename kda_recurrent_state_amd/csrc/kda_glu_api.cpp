// kda_glu_api.cpp -- the extern "C" entry points of the gated feed-forward products
// (include/kda.h): argument validation, workspace, launch.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/kda.h"
#include "kda_checks.hpp"
#include "kda_glu.hpp"

using namespace kda::checks;

namespace {

constexpr int kMaxWidth_ = 1 << 20;

int plan(const kda_glu_dims_t* d, const void* x, const void* w_gate, const void* w_up, kda::GluArgs* a) {
    if (!d) return fail(KDA_ERR_INVALID_ARGUMENT, "dims is NULL");
    if (d->tokens < 0 || d->tokens > kMaxTokens)
        return fail(KDA_ERR_INVALID_ARGUMENT, "tokens = %lld: must be 0 to %lld", (long long)d->tokens, (long long)kMaxTokens);
    if (d->width < 1 || d->width > kMaxWidth_)
        return fail(KDA_ERR_INVALID_ARGUMENT, "width = %d: must be 1 to %d", d->width, kMaxWidth_);
    if (d->hidden < 1 || d->hidden > kMaxWidth_)
        return fail(KDA_ERR_INVALID_ARGUMENT, "hidden = %d: must be 1 to %d", d->hidden, kMaxWidth_);
    KDA_TRY(check_dtype(d->dtype, "dtype"));
    *a = kda::GluArgs();
    switch (d->activation) {
        case KDA_ACT_SILU: a->act = kda::GLU_SILU; break;
        case KDA_ACT_SIGMOID: a->act = kda::GLU_SIGMOID; break;
        case KDA_ACT_GELU: a->act = kda::GLU_GELU; break;
        default:
            return fail(KDA_ERR_INVALID_ARGUMENT, "activation = %d is not KDA_ACT_SILU, KDA_ACT_SIGMOID or KDA_ACT_GELU",
                        d->activation);
    }
    a->T = d->tokens;
    a->D = d->width;
    a->F = d->hidden;
    a->dtype = d->dtype;
    KDA_TRY(check_stride(&a->xs, d->x_stride, a->D, "x_stride"));
    KDA_TRY(check_stride(&a->hs, d->dh_stride, a->F, "dh_stride"));
    const int e = esize(a->dtype);
    const void* ptrs[] = {w_gate, w_up, x};
    const char* names[] = {"w_gate", "w_up", "x"};
    const int align[] = {e, e, e};
    KDA_TRY(check_ptrs(ptrs, names, align, a->T > 0 ? 3 : 2));
    const bool whole = a->dtype == KDA_BF16 && a->D % 64 == 0;
    a->x_plain = whole && (uintptr_t)x % 16 == 0 && a->xs % 8 == 0 && a->xs <= kMaxWidth_;
    a->w_plain = whole && (uintptr_t)w_gate % 16 == 0 && (uintptr_t)w_up % 16 == 0;
    a->x = x;
    a->wg = w_gate;
    a->wu = w_up;
    if (kda::glu_blocks(*a) > 0x7fffff)
        return fail(KDA_ERR_INVALID_ARGUMENT, "tokens, width and hidden = %lld, %d and %d are too large for one launch",
                    (long long)a->T, a->D, a->F);
    return KDA_OK;
}

}  // namespace

extern "C" {

int kda_glu_workspace_size(const kda_glu_dims_t* d, const void* x, const void* w_gate, const void* w_up, int backward,
                           size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARGUMENT, "bytes is NULL");
    kda::GluArgs a;
    KDA_TRY(plan(d, x, w_gate, w_up, &a));
    *bytes = backward ? kda::glu_bwd_workspace(a, true) : kda::glu_fwd_workspace(a);
    return ok();
}

int kda_glu_fwd(const kda_glu_dims_t* d, const void* x, const void* w_gate, const void* w_up, void* h, float* saved,
                void* workspace, size_t workspace_bytes, void* stream) {
    kda::GluArgs a;
    KDA_TRY(plan(d, x, w_gate, w_up, &a));
    if (a.T == 0) return ok();
    const void* ptrs[] = {h};
    const char* names[] = {"h"};
    const int align[] = {esize(a.dtype)};
    KDA_TRY(check_ptrs(ptrs, names, align, 1));
    KDA_TRY(check_optional(saved, 4, "saved"));
    KDA_TRY(check_workspace(workspace, workspace_bytes, kda::glu_fwd_workspace(a)));
    a.h = h;
    a.saved = saved;
    a.ws = static_cast<uint8_t*>(workspace);
    return hip_status(kda::launch_glu_fwd(a, (hipStream_t)stream), "gated products");
}

int kda_glu_bwd(const kda_glu_dims_t* d, const void* x, const void* w_gate, const void* w_up, const float* saved,
                const void* dh, void* dx, void* dw_gate, void* dw_up, void* workspace, size_t workspace_bytes,
                void* stream) {
    kda::GluArgs a;
    KDA_TRY(plan(d, x, w_gate, w_up, &a));
    const int e = esize(a.dtype);
    const void* ptrs[] = {dw_gate, dw_up, dh};
    const char* names[] = {"dw_gate", "dw_up", "dh"};
    const int align[] = {e, e, e};
    KDA_TRY(check_ptrs(ptrs, names, align, a.T > 0 ? 3 : 2));
    KDA_TRY(check_optional(dx, e, "dx"));
    KDA_TRY(check_optional(saved, 4, "saved"));
    KDA_TRY(check_workspace(workspace, workspace_bytes, kda::glu_bwd_workspace(a, dx != nullptr)));
    a.saved = const_cast<float*>(saved);
    a.dh = dh;
    a.dx = dx;
    a.dwg = dw_gate;
    a.dwu = dw_up;
    a.ws = static_cast<uint8_t*>(workspace);
    return hip_status(kda::launch_glu_bwd(a, (hipStream_t)stream), "gated products' gradient");
}

}  // extern "C"
