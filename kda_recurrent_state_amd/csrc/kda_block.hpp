// kda_block.hpp -- host-side launchers of the operators around the state layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// Column sums: out[c] = sum over p of part[p][c], p < rows, c < cols; columns at
// and past split go to out2[c - split].  Either output may be null (skipped).
hipError_t launch_colsum(const float* part, int rows, int64_t cols, int64_t split, float* out, float* out2,
                         hipStream_t st);

struct NormGateArgs {
    const void* x;
    const float* weight;  // may be null (ones)
    const void* gate;     // may be null (no gate)
    const void* dy;       // backward
    void* y;              // forward output, backward: dx
    void* dgate;
    float* part;          // backward: [blocks][width] partial dweight, or null
    int64_t rows;         // tokens x heads
    int32_t heads, width;
    int64_t xs, gs, ds;   // token strides
    float eps;
    int32_t silu;         // gate activation: 1 SiLU, 0 sigmoid
    int32_t dtype;
};
hipError_t launch_norm_gate(const NormGateArgs& a, bool backward, hipStream_t st);
int norm_gate_blocks(int dtype, int width, int64_t rows);  // workgroups (partial rows) of the backward

struct ResNormArgs {
    const void* x;
    const void* res;      // forward: residual in; backward: the stored sum
    const float* weight;
    const float* cscale;  // may be null (ones)
    const void* dy;
    const void* dres;     // may be null (zeros)
    void* res_out;        // forward: the sum; backward: dresidual
    void* y;              // forward: y; backward: dx
    float* part;          // backward: [blocks][width or 2 width] partials (dweight, then dchannel_scale), or null
    int32_t want_dcs;
    int64_t rows;
    int32_t width;
    int64_t xs, rs, ds, drs;
    float eps, scale;
    int32_t dtype, rdtype;
};
hipError_t launch_res_norm(const ResNormArgs& a, bool backward, hipStream_t st);
int res_norm_blocks(const ResNormArgs& a);  // workgroups (partial rows) of the backward

struct ConvArgs {
    const void* x;
    const float* weight;
    const float* bias;    // may be null
    const void* state;    // may be null
    const int32_t* cu;    // device, may be null (equal lengths eq)
    const void* dy;
    const void* dstT;     // may be null
    void* y;              // forward: y; backward: dx
    void* state_T;        // forward: may be null; backward: dstate, may be null
    float* part;          // backward: [rows][C (W + 1)] partials: dweight [C][W], then dbias [C]
    int32_t N, T, eq, C, W;
    int64_t xs, ds;
    int32_t silu, dtype;
};
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t st);
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t st);
int conv_bwd_parts(int T, int N, int C);  // partial rows of the backward
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t st);

struct LinScanArgs {
    const void* x;
    const float* la;
    const float* h0;      // may be null
    const int32_t* cu;    // device, may be null
    const void* dy;
    const float* dhT;     // may be null
    void* y;              // forward: y; backward: dx
    float* dla;
    float* hT;            // forward: may be null; backward: dh0, may be null
    float* states;        // state before every 64th token, [ceil(T / 64)][C]; forward: may be null
    uint64_t* word;       // scratch: linscan_chain_bytes
    int32_t N, T, eq, C;
    int64_t xs, ls, ds;
    int32_t dtype;
};
constexpr int LINSCAN_TILE = 128;  // tokens of the shortest tiles
constexpr int LINSCAN_LINE = 16;  // words of a 128-byte line
// The chain between tiles: one word per tile and channel, and a counter per block
// of 64 channels or more.
inline size_t linscan_chain_bytes(int64_t T, int64_t C) {
    const size_t tiles = (size_t)((T + LINSCAN_TILE - 1) / LINSCAN_TILE);
    return tiles > 1 ? (tiles * C + (C + 63) / 64 * LINSCAN_LINE) * 8 : 0;
}
hipError_t launch_linscan_fwd(const LinScanArgs& a, bool out, hipStream_t st);  // out: y, hT; states where given
hipError_t launch_linscan_bwd(const LinScanArgs& a, hipStream_t st);            // dx, dla, dh0 from states
hipError_t launch_linscan_step(const LinScanArgs& a, hipStream_t st);

}  // namespace kda
