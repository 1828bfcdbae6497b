// kda_glu.hpp -- sizes and host-side launchers of the gated feed-forward products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

enum GluAct { GLU_SILU = 0, GLU_SIGMOID = 1, GLU_GELU = 2 };

// Tokens up to which the forward streams the weights past a few tokens instead of tiling.
constexpr int64_t GLU_FEW = 64;

struct GluArgs {
    const void *x, *wg, *wu, *dh;
    void *h, *dx, *dwg, *dwu;
    float* saved;          // forward: may be null; backward: null to compute again
    int64_t T, xs, hs;     // tokens; token strides of x and dh
    int32_t D, F, dtype, act;
    uint8_t* ws;
    // whether the inputs lie as the tiled kernels read them (bf16, 16-byte rows, whole steps of the sum)
    int32_t x_plain, w_plain;
};

size_t glu_fwd_workspace(const GluArgs& a);
size_t glu_bwd_workspace(const GluArgs& a, bool input_grad);
int64_t glu_blocks(const GluArgs& a);  // workgroups of the largest launch, at most
hipError_t launch_glu_fwd(const GluArgs& a, hipStream_t st);
hipError_t launch_glu_bwd(const GluArgs& a, hipStream_t st);

}  // namespace kda
