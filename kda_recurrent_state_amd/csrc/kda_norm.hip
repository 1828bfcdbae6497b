// kda_norm.hip -- RMS norms around a token-mixing block on gfx950.
//
// norm_gate:      y = x r w s(g),  r = (mean x^2 + eps)^{-1/2},  s a gate activation
//   gradient, with n = x r and d = dy w s(g):
//     dx = r (d - n mean(d n)),  dg = dy n w s'(g),  dw = sum over rows of dy s(g) n
// residual_norm:  h = res + c x,  y = h r(h) w
//   gradient at h, with d = dy w:
//     dh = dres + r (d - n mean(d n)),  dx = c dh,  dw = sum dy n,  dcs = scale sum dh x
//
// All are one pass over HBM: each row is read once into registers, its sums are
// formed over the G lanes (or the whole workgroup) that hold it, and the
// outputs leave from the same registers.  mean(d n) = r mean(d x), so both of
// the backward's sums are formed before r is known and share one reduction.
#include "kda_block.hpp"
#include "kda_rows.hpp"

namespace kda {
namespace {

constexpr int BT = 256;

// Sums of A values over the lanes of a row: G lanes of a wavefront, or (G = BT)
// the whole workgroup through LDS.
template <int G, int A>
__device__ __forceinline__ void row_sum(float (&v)[A], float* lds) {
    if constexpr (G <= WAVE) {
#pragma unroll
        for (int i = 0; i < A; ++i) v[i] = lanes_sum<G>(v[i]);
    } else {
        constexpr int NW = BT / WAVE;
        const int wv = threadIdx.x / WAVE;
        __syncthreads();  // the previous row's sums have been read
#pragma unroll
        for (int i = 0; i < A; ++i) {
            v[i] = lanes_sum<WAVE>(v[i]);
            if (threadIdx.x % WAVE == 0) lds[i * NW + wv] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < A; ++i) {
            v[i] = lds[i * NW];
#pragma unroll
            for (int w = 1; w < NW; ++w) v[i] += lds[i * NW + w];
        }
    }
}

// A workgroup's partial column sums: each of its BT / G row groups holds acc for
// the same columns; summed in group order and written to out[0 .. D).
template <int G, int VPT, int V>
__device__ __forceinline__ void block_partial(const float (&acc)[VPT][V], float* lds, float* out, int D) {
    constexpr int RPB = BT / G, W_ = G * VPT * V;
    const int g = threadIdx.x % G, rg = threadIdx.x / G;
    __syncthreads();
    if constexpr (RPB == 1) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) store_n<float, V>(out + (j * G + g) * V, D - (j * G + g) * V, acc[j]);
    } else {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) lds[rg * W_ + (j * G + g) * V + i] = acc[j][i];
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += BT) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < RPB; ++r) s += lds[r * W_ + c];
            out[c] = s;
        }
    }
}

template <typename T, int V, int G, int VPT>
__global__ __launch_bounds__(BT) void norm_gate_fwd_kernel(NormGateArgs a) {
    constexpr int RPB = BT / G;
    __shared__ float lds[BT / WAVE];
    const int g = threadIdx.x % G, D = a.width;
    const float invD = 1.f / (float)D;
    for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / G; r < a.rows; r += (int64_t)gridDim.x * RPB) {
        const uint32_t t = (uint32_t)r / (uint32_t)a.heads, h = (uint32_t)r - t * a.heads;
        const T* xp = (const T*)a.x + (int64_t)t * a.xs + (int64_t)h * D;
        const T* gp = (const T*)a.gate + (int64_t)t * a.gs + (int64_t)h * D;
        float x[VPT][V], gt[VPT][V], ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * G + g) * V;
            load_n<T, V>(xp + c, D - c, x[j]);
            if (a.gate) load_n<T, V>(gp + c, D - c, gt[j]);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) ss[0] += x[j][i] * x[j][i];
        row_sum<G, 1>(ss, lds);
        const float rn = rsqrtf(ss[0] * invD + a.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * G + g) * V;
            float w[V], y[V];
            if (a.weight) load_n<float, V>(a.weight + c, D - c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                y[i] = x[j][i] * rn;
                if (a.weight) y[i] *= w[i];
                if (a.gate) {
                    const float s = sigmoid_f(gt[j][i]);
                    y[i] *= a.silu ? gt[j][i] * s : s;
                }
            }
            store_n<T, V>((T*)a.y + r * D + c, D - c, y);
        }
    }
}

template <typename T, int V, int G, int VPT>
__global__ __launch_bounds__(BT) void norm_gate_bwd_kernel(NormGateArgs a) {
    constexpr int RPB = BT / G;
    __shared__ float lds[RPB > 1 ? RPB * G * VPT * V : 2 * BT / WAVE];
    const int g = threadIdx.x % G, D = a.width;
    const float invD = 1.f / (float)D;
    float dw[VPT][V] = {};
    for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / G; r < a.rows; r += (int64_t)gridDim.x * RPB) {
        const uint32_t t = (uint32_t)r / (uint32_t)a.heads, h = (uint32_t)r - t * a.heads;
        const T* xp = (const T*)a.x + (int64_t)t * a.xs + (int64_t)h * D;
        const T* gp = (const T*)a.gate + (int64_t)t * a.gs + (int64_t)h * D;
        const T* dp = (const T*)a.dy + (int64_t)t * a.ds + (int64_t)h * D;
        float x[VPT][V], gt[VPT][V], dy[VPT][V], sm[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * G + g) * V;
            load_n<T, V>(xp + c, D - c, x[j]);
            load_n<T, V>(dp + c, D - c, dy[j]);
            if (a.gate) load_n<T, V>(gp + c, D - c, gt[j]);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * G + g) * V;
            float w[V];
            if (a.weight) load_n<float, V>(a.weight + c, D - c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float act = 1.f;
                if (a.gate) {
                    const float s = sigmoid_f(gt[j][i]);
                    act = a.silu ? gt[j][i] * s : s;
                }
                sm[0] += x[j][i] * x[j][i];
                sm[1] += dy[j][i] * act * (a.weight ? w[i] : 1.f) * x[j][i];
            }
        }
        row_sum<G, 2>(sm, lds);
        const float rn = rsqrtf(sm[0] * invD + a.eps);
        const float k = rn * rn * sm[1] * invD;  // r mean(d n)
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * G + g) * V;
            float w[V], dx[V], dg[V];
            if (a.weight) load_n<float, V>(a.weight + c, D - c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float wi = a.weight ? w[i] : 1.f, n = x[j][i] * rn;
                float act = 1.f, slope = 0.f;
                if (a.gate) {
                    const float s = sigmoid_f(gt[j][i]);
                    act = a.silu ? gt[j][i] * s : s;
                    slope = a.silu ? s * (1.f + gt[j][i] * (1.f - s)) : s * (1.f - s);
                }
                dx[i] = rn * (dy[j][i] * act * wi - x[j][i] * k);
                dg[i] = dy[j][i] * n * wi * slope;
                dw[j][i] += dy[j][i] * act * n;
            }
            store_n<T, V>((T*)a.y + r * D + c, D - c, dx);
            if (a.gate) store_n<T, V>((T*)a.dgate + r * D + c, D - c, dg);
        }
    }
    if (a.part) block_partial<G, VPT, V>(dw, lds, a.part + (int64_t)blockIdx.x * D, D);
}

template <typename T, typename R, int V, int G, int VPT>
__global__ __launch_bounds__(BT) void res_norm_fwd_kernel(ResNormArgs a) {
    constexpr int RPB = BT / G;
    __shared__ float lds[BT / WAVE];
    const int g = threadIdx.x % G, D = a.width;
    const float invD = 1.f / (float)D;
    for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / G; r < a.rows; r += (int64_t)gridDim.x * RPB) {
        float h[VPT][V], ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * G + g) * V;
            float x[V], cs[V];
            load_n<R, V>((const R*)a.res + r * a.rs + c, D - c, h[j]);
            load_n<T, V>((const T*)a.x + r * a.xs + c, D - c, x);
            if (a.cscale) load_n<float, V>(a.cscale + c, D - c, cs);
#pragma unroll
            for (int i = 0; i < V; ++i) h[j][i] += (a.cscale ? a.scale * cs[i] : a.scale) * x[i];
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) ss[0] += h[j][i] * h[j][i];
        row_sum<G, 1>(ss, lds);
        const float rn = rsqrtf(ss[0] * invD + a.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * G + g) * V;
            float w[V], y[V];
            load_n<float, V>(a.weight + c, D - c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = h[j][i] * rn * w[i];
            store_n<R, V>((R*)a.res_out + r * D + c, D - c, h[j]);
            store_n<T, V>((T*)a.y + r * D + c, D - c, y);
        }
    }
}

template <typename T, typename R, int V, int G, int VPT>
__global__ __launch_bounds__(BT) void res_norm_bwd_kernel(ResNormArgs a) {
    constexpr int RPB = BT / G;
    __shared__ float lds[RPB > 1 ? RPB * G * VPT * V : 2 * BT / WAVE];
    const int g = threadIdx.x % G, D = a.width;
    const float invD = 1.f / (float)D;
    float dw[VPT][V] = {}, dcs[VPT][V] = {};
    for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / G; r < a.rows; r += (int64_t)gridDim.x * RPB) {
        float h[VPT][V], dy[VPT][V], dr[VPT][V], sm[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * G + g) * V;
            load_n<R, V>((const R*)a.res + r * a.rs + c, D - c, h[j]);
            load_n<T, V>((const T*)a.dy + r * a.ds + c, D - c, dy[j]);
            if (a.dres) load_n<R, V>((const R*)a.dres + r * a.drs + c, D - c, dr[j]);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * G + g) * V;
            float w[V];
            load_n<float, V>(a.weight + c, D - c, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sm[0] += h[j][i] * h[j][i];
                sm[1] += dy[j][i] * w[i] * h[j][i];
            }
        }
        row_sum<G, 2>(sm, lds);
        const float rn = rsqrtf(sm[0] * invD + a.eps);
        const float k = rn * rn * sm[1] * invD;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = (j * G + g) * V;
            float w[V], cs[V], x[V], dx[V], dh[V];
            load_n<float, V>(a.weight + c, D - c, w);
            if (a.cscale) load_n<float, V>(a.cscale + c, D - c, cs);
            if (a.want_dcs) load_n<T, V>((const T*)a.x + r * a.xs + c, D - c, x);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dh[i] = rn * (dy[j][i] * w[i] - h[j][i] * k);
                if (a.dres) dh[i] += dr[j][i];
                dx[i] = (a.cscale ? a.scale * cs[i] : a.scale) * dh[i];
                dw[j][i] += dy[j][i] * h[j][i] * rn;
                if (a.want_dcs) dcs[j][i] += a.scale * dh[i] * x[i];
            }
            store_n<R, V>((R*)a.res_out + r * D + c, D - c, dh);
            store_n<T, V>((T*)a.y + r * D + c, D - c, dx);
        }
    }
    if (a.part) {
        float* out = a.part + (int64_t)blockIdx.x * D * (a.want_dcs ? 2 : 1);
        block_partial<G, VPT, V>(dw, lds, out, D);
        if (a.want_dcs) block_partial<G, VPT, V>(dcs, lds, out + D, D);
    }
}

// Column sums of a [rows][cols] matrix: 16 columns per workgroup, 64 row lanes
// each, so that a narrow matrix still spreads over the rows.
constexpr int CSW = 16, CSR = 64;
__global__ __launch_bounds__(CSW* CSR) void colsum_kernel(const float* part, int rows, int64_t cols, int64_t split,
                                                          float* out, float* out2) {
    __shared__ float lds[CSR][CSW + 1];
    const int cl = threadIdx.x % CSW, rl = threadIdx.x / CSW;
    const int64_t c = (int64_t)blockIdx.x * CSW + cl;
    float s = 0.f;
    if (c < cols)
        for (int r = rl; r < rows; r += CSR) s += part[(int64_t)r * cols + c];
    lds[rl][cl] = s;
#pragma unroll
    for (int k = CSR / 2; k > 0; k >>= 1) {
        __syncthreads();
        if (rl < k) lds[rl][cl] += lds[rl + k][cl];
    }
    if (rl == 0 && c < cols) {
        if (c < split) {
            if (out) out[c] = lds[0][cl];
        } else if (out2) {
            out2[c - split] = lds[0][cl];
        }
    }
}

// Lanes and vectors per lane of a row of nv vectors.
struct RowShape { int g, vpt; };
RowShape row_shape(int nv) {
    if (nv <= 4) return {4, 1};
    if (nv <= 8) return {8, 1};
    if (nv <= 16) return {16, 1};
    if (nv <= 32) return {32, 1};
    if (nv <= 64) return {64, 1};
    if (nv <= 128) return {64, 2};
    if (nv <= 256) return {256, 1};
    if (nv <= 512) return {256, 2};
    if (nv <= 1024) return {256, 4};
    return {256, 8};
}
int vec_of(int dtype) { return dtype == 1 ? 8 : 4; }

int blocks_for(int dtype, int width, int64_t rows, int most) {
    const int v = vec_of(dtype);
    const RowShape s = row_shape((width + v - 1) / v);
    const int64_t rpb = BT / s.g, b = (rows + rpb - 1) / rpb;
    return (int)(b < most ? b : most);
}

constexpr int FWD_BLOCKS = 1 << 20;  // one row group each up to here
constexpr int BWD_BLOCKS = 1024;     // four workgroups per compute unit; each writes one partial row

#define KDA_ROW_CASES(RUN, V)                                                                                  \
    switch (s.g * 16 + s.vpt) {                                                                                \
        case 4 * 16 + 1: RUN(V, 4, 1); break;                                                                  \
        case 8 * 16 + 1: RUN(V, 8, 1); break;                                                                  \
        case 16 * 16 + 1: RUN(V, 16, 1); break;                                                                \
        case 32 * 16 + 1: RUN(V, 32, 1); break;                                                                \
        case 64 * 16 + 1: RUN(V, 64, 1); break;                                                                \
        case 64 * 16 + 2: RUN(V, 64, 2); break;                                                                \
        case 256 * 16 + 1: RUN(V, 256, 1); break;                                                              \
        case 256 * 16 + 2: RUN(V, 256, 2); break;                                                              \
        case 256 * 16 + 4: RUN(V, 256, 4); break;                                                              \
        default: if constexpr (V == 4) { RUN(V, 256, 8); } break;                                              \
    }

template <typename T, int V>
void norm_gate_launch(const NormGateArgs& a, bool backward, int blocks, RowShape s, hipStream_t st) {
#define RUN_NG(V_, G, VPT)                                                                                     \
    if (backward) hipLaunchKernelGGL((norm_gate_bwd_kernel<T, V_, G, VPT>), dim3(blocks), dim3(BT), 0, st, a); \
    else hipLaunchKernelGGL((norm_gate_fwd_kernel<T, V_, G, VPT>), dim3(blocks), dim3(BT), 0, st, a)
    KDA_ROW_CASES(RUN_NG, V)
}

template <typename T, typename R, int V>
void res_norm_launch(const ResNormArgs& a, bool backward, int blocks, RowShape s, hipStream_t st) {
#define RUN_RN(V_, G, VPT)                                                                                       \
    if (backward) hipLaunchKernelGGL((res_norm_bwd_kernel<T, R, V_, G, VPT>), dim3(blocks), dim3(BT), 0, st, a); \
    else hipLaunchKernelGGL((res_norm_fwd_kernel<T, R, V_, G, VPT>), dim3(blocks), dim3(BT), 0, st, a)
    KDA_ROW_CASES(RUN_RN, V)
}

}  // namespace

hipError_t launch_colsum(const float* part, int rows, int64_t cols, int64_t split, float* out, float* out2,
                         hipStream_t st) {
    hipLaunchKernelGGL(colsum_kernel, dim3((unsigned)((cols + CSW - 1) / CSW)), dim3(CSW * CSR), 0, st, part, rows,
                       cols, split, out, out2);
    return hipGetLastError();
}

int norm_gate_blocks(int dtype, int width, int64_t rows) { return blocks_for(dtype, width, rows, BWD_BLOCKS); }

hipError_t launch_norm_gate(const NormGateArgs& a, bool backward, hipStream_t st) {
    const int v = vec_of(a.dtype);
    const RowShape s = row_shape((a.width + v - 1) / v);
    const int blocks = blocks_for(a.dtype, a.width, a.rows, backward ? BWD_BLOCKS : FWD_BLOCKS);
    if (a.dtype == 1) norm_gate_launch<bf16, 8>(a, backward, blocks, s, st);
    else norm_gate_launch<float, 4>(a, backward, blocks, s, st);
    return hipGetLastError();
}

int res_norm_blocks(int dtype, int width, int64_t rows) { return blocks_for(dtype, width, rows, BWD_BLOCKS); }

hipError_t launch_res_norm(const ResNormArgs& a, bool backward, hipStream_t st) {
    const int v = vec_of(a.dtype);
    const RowShape s = row_shape((a.width + v - 1) / v);
    const int blocks = blocks_for(a.dtype, a.width, a.rows, backward ? BWD_BLOCKS : FWD_BLOCKS);
    if (a.dtype == 1 && a.rdtype == 1) res_norm_launch<bf16, bf16, 8>(a, backward, blocks, s, st);
    else if (a.dtype == 1) res_norm_launch<bf16, float, 8>(a, backward, blocks, s, st);
    else res_norm_launch<float, float, 4>(a, backward, blocks, s, st);
    return hipGetLastError();
}

}  // namespace kda
