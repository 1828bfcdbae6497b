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
// The launch for T tokens of C channels: vec channels a lane, waves wavefronts of 16
// tokens to a tile, tiles x cblocks workgroups, and up to LINSCAN_EMPTY more for empty
// sequences.
constexpr int LINSCAN_EMPTY = 64;
struct LinScanShape { int vec, waves, tiles, cblocks; };
inline LinScanShape linscan_shape(int32_t T, int32_t C) {
    LinScanShape s;
    s.vec = C < 2 ? 1 : 2;
    // A chain is narrow below 32 column blocks.  Its tiles wait for each other more
    // than for memory, so they are longer: 256 tokens on 16 wavefronts.  In a wide one
    // 128 on 8 leave room for two workgroups on a compute unit, one loading while
    // the other waits or stores.  Measured in a graph, 256 against 128, us: 60000 x 64
    // in one sequence 44 and 75, in 64 sequences 19.4 and 22.9, 4096 x 2048 bf16 20.6 and
    // 22.4, 24571 x 1000 fp32 72 and 75; 2 x 32768 x 4096 bf16 482 and 412, 24571 x 4096
    // fp32 239 and 219.  Between them the length counts as well, which the rule leaves
    // out: 4096 x 3584 bf16 33.3 and 33.6 and its gradient in fp32 90 and 95, but
    // 32768 x 3584 237 and 192, 668 and 592, and 32768 x 2048 137 and 120, 379 and 358.
    s.waves = s.vec == 1 || C < 32 * 64 * s.vec ? 16 : 8;
    s.tiles = (T + s.waves * 16 - 1) / (s.waves * 16);
    s.cblocks = (C + 64 * s.vec - 1) / (64 * s.vec);
    return s;
}
// Whether such a launch stays below 2^32 threads.  One column block of tiles of 256
// is the tightest: n = ceil(T / 128) makes ceil(n / 2) + 64 workgroups of 1024 threads, at
// most 512 n + 66048.  Every other shape has fewer threads for its n column blocks of 64.
inline bool linscan_fits(int64_t T, int64_t C) {
    return (T + LINSCAN_TILE - 1) / LINSCAN_TILE * ((C + 63) / 64) < (1ll << 32) / 512 - 129;
}
hipError_t launch_linscan_fwd(const LinScanArgs& a, bool out, hipStream_t st);  // out: y, hT; states where given
hipError_t launch_linscan_bwd(const LinScanArgs& a, hipStream_t st);            // dx, dla, dh0 from states
hipError_t launch_linscan_step(const LinScanArgs& a, hipStream_t st);

}  // namespace kda
