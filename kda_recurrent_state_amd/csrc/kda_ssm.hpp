// kda_ssm.hpp -- sizes and host-side launchers of the selective state space scan.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// A head's state [K, P] is taken in blocks of all K rows and some columns: columns do not meet in the recurrence.
// The walk along the tokens holds one in a wavefront's registers, 32 columns (16 above 128 rows); the
// gradient, which reads the states, takes twice as many at a time.  A head's block of columns is a "unit".
constexpr int SSM_MAX_STATE = 256;
inline int ssm_cols(int K) { return K > 128 ? 32 : 64; }
inline int ssm_rows(int K) { return K <= 32 ? 32 : K <= 64 ? 64 : K <= 128 ? 128 : 256; }
inline int ssm_chunk(int dtype) { return dtype == 1 ? 64 : 32; }  // tokens of the gradient's chunk (1: bf16)

struct SsmArgs {
    const void *x, *B, *C, *dy;
    const float *dt, *A, *D, *bias, *h0, *dhT;  // D, bias, h0, dhT may be null
    const int32_t* cu;                           // device, may be null
    void *y, *dB, *dC;                           // y: forward output; backward: dx
    float *hT, *ddt, *dA, *dD, *dbias, *dh0;     // each may be null but ddt
    int32_t N, T, eq, H, G, K, P;
    int64_t xs, dts, bs, cs, dys;                // token strides
    int32_t dtype, softplus;
    // plan
    int32_t chunk, rows;                         // tokens of a chunk, padded K
    int32_t cols, blocks, wcols, wblocks;        // columns of a block, blocks of a head: of the gradient, of the walk
    int32_t seg;                                 // tokens of a segment (a multiple of chunk)
    int32_t split;                               // shares of a group's units in the gradient
    // workspace
    float *ends, *decay;                         // a segment's own state at its end / the state it starts from; its decay
    float *rends, *rdecay;                       // the same of the gradient's reverse walk
    float *hs, *gs;                              // states before every chunk, derivatives behind it
    float *part;                                 // partial dB, dC of the shares
    float *dec;                                  // decays of every chunk and head
    float *tok;                                  // numbers of every chunk's tokens and unit
    float *sums;                                 // every chunk's parts of dA, dD, dbias
};

inline int64_t ssm_units(const SsmArgs& a) { return (int64_t)a.H * a.blocks; }
inline int64_t ssm_slots(const SsmArgs& a, int every) { return (int64_t)a.T / every + a.N; }
inline int64_t ssm_unit_state(const SsmArgs& a) { return (int64_t)a.rows * a.cols; }  // of the gradient's units
constexpr int ssm_token_floats(int chunk) { return 7 * chunk + 16; }  // of a chunk and unit
inline int64_t ssm_decay_floats(const SsmArgs& a) { return 5ll * a.chunk + 16; }

hipError_t launch_ssm_fwd(const SsmArgs& a, hipStream_t st);
hipError_t launch_ssm_bwd(const SsmArgs& a, hipStream_t st);

struct SsmStepArgs {
    const void *x, *B, *C;      // in: dtype; with a convolution all three lie in conv's float output
    const float *dt, *A, *D, *bias, *h_in;
    float* h_out;
    void* y;
    int32_t N, H, G, K, P;
    int64_t xs, dts, bs, cs;
    int32_t dtype, softplus, f32_in;
};
hipError_t launch_ssm_step(const SsmStepArgs& a, hipStream_t st);

struct SsmConvArgs {
    const void* x;
    const float *weight, *bias;  // bias may be null
    const void* state_in;
    void* state_out;
    float* z;                    // [N, C]
    int32_t N, C, W, dtype, silu;
    int64_t xs;
};
hipError_t launch_ssm_conv(const SsmConvArgs& a, hipStream_t st);

}  // namespace kda
