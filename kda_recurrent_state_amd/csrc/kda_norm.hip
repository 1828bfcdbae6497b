// kda_norm.hip -- RMS norms around a token-mixing block on gfx950.
//
// norm_gate:      y = x r w s(g),  r = (mean x^2 + eps)^{-1/2},  s a gate activation
//   gradient, with n = x r and d = dy w s(g):
//     dx = r (d - n mean(d n)),  dg = dy n w s'(g),  dw = sum over rows of dy s(g) n
// residual_norm:  h = res + c x,  y = h r(h) w
//   gradient at h, with d = dy w:
//     dh = dres + r (d - n mean(d n)),  dx = c dh,  dw = sum dy n,  dcs = scale sum dh x
//
// All are one pass over HBM, which bounds them (5.5 to 6 TB/s on large inputs): each
// row is read once into registers, its sums are formed over the G lanes (or the
// whole workgroup) that hold it, and the outputs leave from the same registers.
// mean(d n) = r mean(d x), so both of the backward's sums are formed before r is
// known and share one reduction.
#include "kda_block.hpp"
#include "kda_rows.hpp"

namespace kda {
namespace {

// Threads of a workgroup whose rows take G lanes: 256, or one row's G.
constexpr int threads_of(int g) { return g > 256 ? g : 256; }

// Sums of A values over the lanes of a row: G lanes of a wavefront, or (G >= 256)
// the whole workgroup through LDS.
template <int G, int A>
__device__ __forceinline__ void row_sum(float (&v)[A], float* lds) {
    if constexpr (G <= WAVE) {
#pragma unroll
        for (int i = 0; i < A; ++i) v[i] = lanes_sum<G>(v[i]);
    } else {
        constexpr int NW = G / WAVE;
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

// The columns of a lane's j-th vector: first column c (the row's last V where the
// vector would pass its end), and how many of them (0 to V) a neighbour or
// nobody counts; lanes past the row's end have V and store nothing.
template <int V, int G> struct Cols {
    int c, skip;
    bool live;
    __device__ __forceinline__ Cols(int j, int g, int D) {
        const int at = (j * G + g) * V;
        c = column<V>(at, D);
        skip = at - c < V ? at - c : V;
        live = at < D;
    }
};

// A workgroup's partial column sums: each of its row groups holds acc for
// the same columns; summed in group order and written to out[0 .. D).
template <int G, int VPT, int V>
__device__ __forceinline__ void block_partial(const float (&acc)[VPT][V], float* lds, float* out, int D) {
    constexpr int BT = threads_of(G), RPB = BT / G, W_ = G * VPT * V;
    const int g = threadIdx.x % G, rg = threadIdx.x / G;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const Cols<V, G> cl(j, g, D);
        if (!cl.live) continue;
        if constexpr (RPB == 1) {
            store_v<V>(out + cl.c, acc[j]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) lds[rg * W_ + cl.c + i] = acc[j][i];
        }
    }
    if constexpr (RPB > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += BT) {
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < RPB; ++r) s += lds[r * W_ + c];
            out[c] = s;
        }
    }
}

// The gate: none, a logistic function of it, or it times that.  s is its
// logistic value.
enum { GATE_NONE, GATE_SIGMOID, GATE_SILU };
template <int GATE> __device__ __forceinline__ float gate_act(float g, float s) {
    return GATE == GATE_SILU ? g * s : GATE == GATE_SIGMOID ? s : 1.f;
}
// The logistic slope is as small as the smaller of s and 1 - s, and as right: for g > 0 the
// difference would lose it (all of it from g = 17 on), e^-g s is the same number.  SiLU's
// slope is near 1 there, which 1 - s is as right as it has to be for.
template <int GATE> __device__ __forceinline__ float gate_slope(float g, float s) {
    return GATE == GATE_SILU ? s * (1.f + g * (1.f - s)) : s * (g > 0.f ? __expf(-g) * s : 1.f - s);
}

template <typename T, int V, int G, int VPT, int GATE, bool PAST>
__global__ __launch_bounds__(threads_of(G)) void norm_gate_fwd_kernel(NormGateArgs a) {
    constexpr int BT = threads_of(G), RPB = BT / G;
    __shared__ float lds[BT / WAVE];
    const int g = threadIdx.x % G, D = a.width;
    const float invD = 1.f / (float)D;
    const T* x = (const T*)a.x;
    const T* gate = (const T*)a.gate;
    for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / G; r < a.rows; r += (int64_t)gridDim.x * RPB) {
        const uint32_t t = (uint32_t)r / (uint32_t)a.heads, h = (uint32_t)r - t * a.heads;
        const T* xp = x + (int64_t)t * a.xs + (int64_t)h * D;
        const T* gp = gate + (int64_t)t * a.gs + (int64_t)h * D;
        Pack<T, V> xr[VPT], gr[VPT];
        Pack<float, V> wr[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) xr[j] = load_c<PAST, V>(xp + Cols<V, G>(j, g, D).c);
        if (GATE)
#pragma unroll
            for (int j = 0; j < VPT; ++j) gr[j] = load_c<PAST, V>(gp + Cols<V, G>(j, g, D).c);
        if (a.weight)
#pragma unroll
            for (int j = 0; j < VPT; ++j) wr[j] = load_v<V>(a.weight + Cols<V, G>(j, g, D).c);
        float ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const Cols<V, G> cl(j, g, D);
#pragma unroll
            for (int i = 0; i < V; ++i) ss[0] += i >= cl.skip ? xr[j][i] * xr[j][i] : 0.f;
        }
        row_sum<G, 1>(ss, lds);
        const float rn = rsqrtf(ss[0] * invD + a.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const Cols<V, G> cl(j, g, D);
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = xr[j][i] * rn;
            if (a.weight)
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] *= wr[j][i];
            if (GATE)
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] *= gate_act<GATE>(gr[j][i], sigmoid_f(gr[j][i]));
            if (cl.live) store_c<PAST, V>((T*)a.y + r * D + cl.c, y);
        }
    }
}

template <typename T, int V, int G, int VPT, int GATE, bool PAST>
__global__ __launch_bounds__(threads_of(G)) void norm_gate_bwd_kernel(NormGateArgs a) {
    constexpr int BT = threads_of(G), RPB = BT / G;
    __shared__ float lds[RPB > 1 ? RPB * G * VPT * V : 2 * BT / WAVE];
    const int g = threadIdx.x % G, D = a.width;
    const float invD = 1.f / (float)D;
    const T* x = (const T*)a.x;
    const T* gate = (const T*)a.gate;
    const T* dyb = (const T*)a.dy;
    float w[VPT][V], dw[VPT][V] = {};
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) w[j][i] = a.weight ? a.weight[Cols<V, G>(j, g, D).c + i] : 1.f;
    for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / G; r < a.rows; r += (int64_t)gridDim.x * RPB) {
        const uint32_t t = (uint32_t)r / (uint32_t)a.heads, h = (uint32_t)r - t * a.heads;
        const T* xp = x + (int64_t)t * a.xs + (int64_t)h * D;
        const T* gp = gate + (int64_t)t * a.gs + (int64_t)h * D;
        const T* dp = dyb + (int64_t)t * a.ds + (int64_t)h * D;
        Pack<T, V> xr[VPT], gr[VPT], dr[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = Cols<V, G>(j, g, D).c;
            xr[j] = load_c<PAST, V>(xp + c);
            dr[j] = load_c<PAST, V>(dp + c);
        }
        if (GATE)
#pragma unroll
            for (int j = 0; j < VPT; ++j) gr[j] = load_c<PAST, V>(gp + Cols<V, G>(j, g, D).c);
        float sg[VPT][V], sm[2] = {0.f, 0.f};  // sg: the gate's logistic value
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const Cols<V, G> cl(j, g, D);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sg[j][i] = GATE ? sigmoid_f(gr[j][i]) : 1.f;
                const float act = GATE ? gate_act<GATE>(gr[j][i], sg[j][i]) : 1.f;
                sm[0] += i >= cl.skip ? xr[j][i] * xr[j][i] : 0.f;
                sm[1] += i >= cl.skip ? dr[j][i] * act * w[j][i] * xr[j][i] : 0.f;
            }
        }
        row_sum<G, 2>(sm, lds);
        const float rn = rsqrtf(sm[0] * invD + a.eps);
        const float k = rn * rn * sm[1] * invD;  // r mean(d n)
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const Cols<V, G> cl(j, g, D);
            float dx[V], dg[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float n = xr[j][i] * rn, dy = dr[j][i];
                const float act = GATE ? gate_act<GATE>(gr[j][i], sg[j][i]) : 1.f;
                dx[i] = rn * (dy * act * w[j][i] - xr[j][i] * k);
                if (GATE) dg[i] = dy * n * w[j][i] * gate_slope<GATE>(gr[j][i], sg[j][i]);
                dw[j][i] += dy * act * n;
            }
            if (cl.live) {
                store_c<PAST, V>((T*)a.y + r * D + cl.c, dx);
                if (GATE) store_c<PAST, V>((T*)a.dgate + r * D + cl.c, dg);
            }
        }
    }
    if (a.part) block_partial<G, VPT, V>(dw, lds, a.part + (int64_t)blockIdx.x * D, D);
}

template <typename T, typename R, int V, int G, int VPT, bool PAST>
__global__ __launch_bounds__(threads_of(G)) void res_norm_fwd_kernel(ResNormArgs a) {
    constexpr int BT = threads_of(G), RPB = BT / G;
    __shared__ float lds[BT / WAVE];
    const int g = threadIdx.x % G, D = a.width;
    const float invD = 1.f / (float)D;
    for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / G; r < a.rows; r += (int64_t)gridDim.x * RPB) {
        Pack<R, V> rr[VPT];
        Pack<T, V> xr[VPT];
        Pack<float, V> wr[VPT], cr[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = Cols<V, G>(j, g, D).c;
            rr[j] = load_c<PAST, V>((const R*)a.res + r * a.rs + c);
            xr[j] = load_c<PAST, V>((const T*)a.x + r * a.xs + c);
        }
#pragma unroll
        for (int j = 0; j < VPT; ++j) wr[j] = load_v<V>(a.weight + Cols<V, G>(j, g, D).c);
        if (a.cscale)
#pragma unroll
            for (int j = 0; j < VPT; ++j) cr[j] = load_v<V>(a.cscale + Cols<V, G>(j, g, D).c);
        float h[VPT][V], ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const Cols<V, G> cl(j, g, D);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                h[j][i] = rr[j][i] + (a.cscale ? a.scale * cr[j][i] : a.scale) * xr[j][i];
                ss[0] += i >= cl.skip ? h[j][i] * h[j][i] : 0.f;
            }
        }
        row_sum<G, 1>(ss, lds);
        const float rn = rsqrtf(ss[0] * invD + a.eps);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const Cols<V, G> cl(j, g, D);
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i) y[i] = h[j][i] * rn * wr[j][i];
            if (cl.live) {
                store_c<PAST, V>((R*)a.res_out + r * D + cl.c, h[j]);
                store_c<PAST, V>((T*)a.y + r * D + cl.c, y);
            }
        }
    }
}

template <typename T, typename R, int V, int G, int VPT, bool PAST>
__global__ __launch_bounds__(threads_of(G)) void res_norm_bwd_kernel(ResNormArgs a) {
    constexpr int BT = threads_of(G), RPB = BT / G;
    __shared__ float lds[RPB > 1 ? RPB * G * VPT * V : 2 * BT / WAVE];
    const int g = threadIdx.x % G, D = a.width;
    const float invD = 1.f / (float)D;
    float w[VPT][V], cs[VPT][V], dw[VPT][V] = {}, dcs[VPT][V] = {};
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = Cols<V, G>(j, g, D).c + i;
            w[j][i] = a.weight[c];
            cs[j][i] = a.cscale ? a.scale * a.cscale[c] : a.scale;
        }
    for (int64_t r = (int64_t)blockIdx.x * RPB + threadIdx.x / G; r < a.rows; r += (int64_t)gridDim.x * RPB) {
        Pack<R, V> hr[VPT], rr[VPT];
        Pack<T, V> dr[VPT], xr[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int c = Cols<V, G>(j, g, D).c;
            hr[j] = load_c<PAST, V>((const R*)a.res + r * a.rs + c);
            dr[j] = load_c<PAST, V>((const T*)a.dy + r * a.ds + c);
        }
        if (a.dres)
#pragma unroll
            for (int j = 0; j < VPT; ++j) rr[j] = load_c<PAST, V>((const R*)a.dres + r * a.drs + Cols<V, G>(j, g, D).c);
        if (a.want_dcs)
#pragma unroll
            for (int j = 0; j < VPT; ++j) xr[j] = load_c<PAST, V>((const T*)a.x + r * a.xs + Cols<V, G>(j, g, D).c);
        float sm[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const Cols<V, G> cl(j, g, D);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sm[0] += i >= cl.skip ? hr[j][i] * hr[j][i] : 0.f;
                sm[1] += i >= cl.skip ? dr[j][i] * w[j][i] * hr[j][i] : 0.f;
            }
        }
        row_sum<G, 2>(sm, lds);
        const float rn = rsqrtf(sm[0] * invD + a.eps);
        const float k = rn * rn * sm[1] * invD;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const Cols<V, G> cl(j, g, D);
            float dx[V], dh[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dh[i] = rn * (dr[j][i] * w[j][i] - hr[j][i] * k);
                if (a.dres) dh[i] += rr[j][i];
                dx[i] = cs[j][i] * dh[i];
                dw[j][i] += dr[j][i] * hr[j][i] * rn;
                if (a.want_dcs) dcs[j][i] += a.scale * dh[i] * xr[j][i];
            }
            if (cl.live) {
                store_c<PAST, V>((R*)a.res_out + r * D + cl.c, dh);
                store_c<PAST, V>((T*)a.y + r * D + cl.c, dx);
            }
        }
    }
    if (a.part) {
        float* out = a.part + (int64_t)blockIdx.x * D * (a.want_dcs ? 2 : 1);
        block_partial<G, VPT, V>(dw, lds, out, D);
        if (a.want_dcs) block_partial<G, VPT, V>(dcs, lds, out + D, D);
    }
}

// Column sums of a [rows][cols] matrix: 16 columns per workgroup, 64 row lanes
// each, so that a narrow matrix still spreads over the rows.  In float32 as the partial
// rows are: a sum over a million rows of 128 is a chain of at most 114 additions (86 rows of a
// group, 16 groups of a workgroup, 12 partial rows) and a tree, so within 121 2^-24 of its
// terms' magnitudes.
constexpr int CSW = 16, CSR = 64;
__global__ __launch_bounds__(CSW* CSR) void colsum_kernel(const float* part, int rows, int64_t cols, int64_t split,
                                                          float* out, float* out2) {
    __shared__ float lds[CSR][CSW + 1];
    const int cl = threadIdx.x % CSW, rl = threadIdx.x / CSW;
    const int64_t c = (int64_t)blockIdx.x * CSW + cl;
    float s = 0.f;
    if (c < cols) {
        int r = rl;
        for (; r + 3 * CSR < rows; r += 4 * CSR) {  // four loads in flight
            const float* q = part + (int64_t)r * cols + c;
            const float v0 = q[0], v1 = q[CSR * cols], v2 = q[2 * CSR * cols], v3 = q[3 * CSR * cols];
            s += (v0 + v1) + (v2 + v3);
        }
        for (; r < rows; r += CSR) s += part[(int64_t)r * cols + c];
    }
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

// Lanes and vectors per lane of a row of nv vectors: a wavefront or part of it up to
// two vectors a lane, longer rows a workgroup.  Measured through the cache, bf16, 64e6 values, forward and
// gradient in us: rows of 1024 as here 92 and 128, over 256 lanes 92 and 223; 2048
// here 93 and 132, a wavefront with four a lane 92 and 132; 4096 here 94, over 512
// lanes 92; 8192 here 97 and 137, 256 lanes with four 95 and 149.
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
    if (nv <= 1024) return {512, 2};
    return {512, 4};
}
// Elements per lane and access: 16 bytes of the row's type, single elements in
// rows shorter than that.
int vec_of(int dtype, int width) {
    const int v = dtype == 1 ? 8 : 4;
    return width >= v ? v : 1;
}

int vecs_of(int dtype, int width) {
    const int v = vec_of(dtype, width);
    return (width + v - 1) / v;
}

// Workgroups of `rows` rows of nv vectors, at most `most`.
int blocks_for(int nv, int64_t rows, int most) {
    const RowShape s = row_shape(nv);
    const int64_t rpb = threads_of(s.g) / s.g, b = (rows + rpb - 1) / rpb;
    return (int)(b < most ? b : most);
}

constexpr int FWD_BLOCKS = 1 << 20;  // one row group each up to here
// The backward's workgroups, a whole number for each of the 256 compute units,
// each of which leaves a partial row: as few as keep enough loads in flight.  Of
// 256, 512, 768 and 1024 took, in us,
//   gated norm, bf16:     32768 x 32 rows of 128: 473, 284, 239, 243;  30000 of 2048: 272, 157, 125, 117
//                         20000 of 4096: 243, 167, 159, 180;  8192 of 8192: 150, 154, 160, 164
//   residual norm, loads  24 KB a row (bf16, 16384 of 4096): 152, 121, 136, 125;  40 KB: 210, 189, 205, 195
//                         48 KB (fp32 stream, 16384 of 4096): 229, 225, 249, 241;  (bf16, 8192 of 8192): 137,
//                         142, 149, 156;  64 KB: 165, 178, 193, 205;  fp32, 20000 rows of 1000: 125, 75, 77, 82
// Both rules split where the figures do, and lie between rows that want either: the gated
// norm's 4096 columns lose 5 % by 512 where its 8192 gain 4 %, the residual norm's two rows
// of 48 KB lose 2 % and gain 4 % by 256.
int ng_blocks(int nv) { return nv > 256 ? 512 : 768; }
int rn_blocks(const ResNormArgs& a) {
    const int e = a.dtype == 1 ? 2 : 4, er = a.rdtype == 1 ? 2 : 4;
    return a.width * (2 * er + e + (a.want_dcs ? e : 0)) >= 48 * 1024 ? 256 : 512;
}

#define KDA_ROW_CASES(RUN, V)                                                                                  \
    switch (s.g * 16 + s.vpt) {                                                                                \
        case 4 * 16 + 1: RUN(V, 4, 1); break;                                                                  \
        case 8 * 16 + 1: if constexpr (V > 1 || sizeof(T) == 2) { RUN(V, 8, 1); } break;                       \
        default: if constexpr (V > 1) KDA_WIDE_CASES(RUN, V) break;                                            \
    }
#define KDA_WIDE_CASES(RUN, V)                                                                                 \
    switch (s.g * 16 + s.vpt) {                                                                                \
        case 16 * 16 + 1: RUN(V, 16, 1); break;                                                                \
        case 32 * 16 + 1: RUN(V, 32, 1); break;                                                                \
        case 64 * 16 + 1: RUN(V, 64, 1); break;                                                                \
        case 64 * 16 + 2: RUN(V, 64, 2); break;                                                                \
        case 256 * 16 + 1: RUN(V, 256, 1); break;                                                              \
        case 256 * 16 + 2: RUN(V, 256, 2); break;                                                              \
        case 512 * 16 + 2: RUN(V, 512, 2); break;                                                              \
        default: if constexpr (V == 4) { RUN(V, 512, 4); }                                                     \
    }

#define KDA_LAUNCH(KERNEL, G, ...) \
    hipLaunchKernelGGL((KERNEL<__VA_ARGS__>), dim3(blocks), dim3(threads_of(G)), 0, st, a)
template <typename T, int V, bool PAST>
void norm_gate_launch(const NormGateArgs& a, bool backward, int blocks, RowShape s, hipStream_t st) {
#define RUN_NG1(V_, G, VPT, GATE)                                                   \
    if (backward) KDA_LAUNCH(norm_gate_bwd_kernel, G, T, V_, G, VPT, GATE, PAST);   \
    else KDA_LAUNCH(norm_gate_fwd_kernel, G, T, V_, G, VPT, GATE, PAST)
#define RUN_NG(V_, G, VPT)                               \
    if (!a.gate) { RUN_NG1(V_, G, VPT, GATE_NONE); }     \
    else if (a.silu) { RUN_NG1(V_, G, VPT, GATE_SILU); } \
    else { RUN_NG1(V_, G, VPT, GATE_SIGMOID); }
    KDA_ROW_CASES(RUN_NG, V)
}
template <typename T, int V>
void norm_gate_launch(const NormGateArgs& a, bool backward, int blocks, RowShape s, bool past, hipStream_t st) {
    if (V > 1 && past) norm_gate_launch<T, V, (V > 1)>(a, backward, blocks, s, st);
    else norm_gate_launch<T, V, false>(a, backward, blocks, s, st);
}

template <typename T, typename R, int V, bool PAST>
void res_norm_launch(const ResNormArgs& a, bool backward, int blocks, RowShape s, hipStream_t st) {
#define RUN_RN(V_, G, VPT)                                                      \
    if (backward) KDA_LAUNCH(res_norm_bwd_kernel, G, T, R, V_, G, VPT, PAST);   \
    else KDA_LAUNCH(res_norm_fwd_kernel, G, T, R, V_, G, VPT, PAST)
    KDA_ROW_CASES(RUN_RN, V)
}
template <typename T, typename R, int V>
void res_norm_launch(const ResNormArgs& a, bool backward, int blocks, RowShape s, bool past, hipStream_t st) {
    if (V > 1 && past) res_norm_launch<T, R, V, (V > 1)>(a, backward, blocks, s, st);
    else res_norm_launch<T, R, V, false>(a, backward, blocks, s, st);
}

}  // namespace

hipError_t launch_colsum(const float* part, int rows, int64_t cols, int64_t split, float* out, float* out2,
                         hipStream_t st) {
    hipLaunchKernelGGL(colsum_kernel, dim3((unsigned)((cols + CSW - 1) / CSW)), dim3(CSW * CSR), 0, st, part, rows,
                       cols, split, out, out2);
    return hipGetLastError();
}

int norm_gate_blocks(int dtype, int width, int64_t rows) {
    const int nv = vecs_of(dtype, width);
    return blocks_for(nv, rows, ng_blocks(nv));
}

hipError_t launch_norm_gate(const NormGateArgs& a, bool backward, hipStream_t st) {
    const int v = vec_of(a.dtype, a.width);
    const int nv = vecs_of(a.dtype, a.width);
    const RowShape s = row_shape(nv);
    const int blocks = blocks_for(nv, a.rows, backward ? ng_blocks(nv) : FWD_BLOCKS);
    const int64_t size = a.rows * a.width * (a.dtype == 1 ? 2 : 4);  // of a tensor
    const bool past = past_cache(size * (1 + backward + (a.gate != nullptr)));
    if (a.dtype == 1 && v == 1) norm_gate_launch<bf16, 1>(a, backward, blocks, s, past, st);
    else if (a.dtype == 1) norm_gate_launch<bf16, 8>(a, backward, blocks, s, past, st);
    else if (v == 1) norm_gate_launch<float, 1>(a, backward, blocks, s, past, st);
    else norm_gate_launch<float, 4>(a, backward, blocks, s, past, st);
    return hipGetLastError();
}

int res_norm_blocks(const ResNormArgs& a) { return blocks_for(vecs_of(a.dtype, a.width), a.rows, rn_blocks(a)); }

hipError_t launch_res_norm(const ResNormArgs& a, bool backward, hipStream_t st) {
    const int v = vec_of(a.dtype, a.width);
    const int nv = vecs_of(a.dtype, a.width);
    const RowShape s = row_shape(nv);
    const int blocks = backward ? res_norm_blocks(a) : blocks_for(nv, a.rows, FWD_BLOCKS);
    const int64_t n = a.rows * a.width, size = n * (a.dtype == 1 ? 2 : 4), rsize = n * (a.rdtype == 1 ? 2 : 4);
    const bool past = past_cache(size + rsize + (backward && a.dres ? rsize : 0) + (backward && a.want_dcs ? size : 0));
    if (v == 1) {
        if (a.dtype == 1 && a.rdtype == 1) res_norm_launch<bf16, bf16, 1>(a, backward, blocks, s, past, st);
        else if (a.dtype == 1) res_norm_launch<bf16, float, 1>(a, backward, blocks, s, past, st);
        else res_norm_launch<float, float, 1>(a, backward, blocks, s, past, st);
    } else {
        if (a.dtype == 1 && a.rdtype == 1) res_norm_launch<bf16, bf16, 8>(a, backward, blocks, s, past, st);
        else if (a.dtype == 1) res_norm_launch<bf16, float, 8>(a, backward, blocks, s, past, st);
        else res_norm_launch<float, float, 4>(a, backward, blocks, s, past, st);
    }
    return hipGetLastError();
}

}  // namespace kda
