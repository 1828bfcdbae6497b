// kda_conv.hip -- short causal depthwise convolution over packed sequences on gfx950.
//
//   z_t[c] = b[c] + sum_{j < W} w[c][j] x_{t-W+1+j}[c],   y_t = z_t or z_t / (1 + e^{-z_t})
//
// where a sequence's tokens are preceded by the W - 1 rows of its state.  The
// gradient, with dz_t = dy_t act'(z_t) and dz = 0 outside a sequence's tokens,
// over its rows s (state rows and tokens alike):
//   dx_s = sum_{k < W} w[W-1-k] dz_{s+k},   dw[W-1-k] = sum_s x_s dz_{s+k},   db = sum_t dz_t,
// plus the derivative of the outgoing state for the rows that form it.
//
// HBM-bound: a thread owns V adjacent channels of a strip of consecutive tokens
// and slides the W-token window along it in registers, so every row is read
// once and the strip's W - 1 leading rows (backward: 2 (W - 1)) once more,
// from cache.  Groups of 8 tokens are loaded together ahead of their use.
// Groups that a sequence's edge crosses take a path of their own, which
// fetches each tap where the sequence says it is.
#include "kda_block.hpp"
#include "kda_rows.hpp"

namespace kda {
namespace {

constexpr int BT = 256;
constexpr int GRP = 8;  // tokens loaded together

__device__ __forceinline__ float act_f(float z, int silu) { return silu ? z * sigmoid_f(z) : z; }

// One thread's view: V channels from c of the packed rows of x and the states.
template <typename T, int V, int W>
struct Taps {
    const T* x;      // channel c of token 0
    const T* state;  // channel c of state row 0, or null
    int64_t xs;
    int C, n_valid;
    // row `pos` (from -(W-1)) of sequence n whose tokens start at beg
    __device__ __forceinline__ void row(int n, int beg, int pos, float (&v)[V]) const {
        if (pos >= 0) {
            load_n<T, V>(x + (int64_t)(beg + pos) * xs, n_valid, v);
        } else if (state) {
            load_n<T, V>(state + ((int64_t)n * (W - 1) + (W - 1 + pos)) * C, n_valid, v);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = 0.f;
        }
    }
};

template <typename T, int V, int W>
__global__ __launch_bounds__(BT) void conv_fwd_kernel(ConvArgs a, int G, int L, int strip_blocks) {
    const Seqs sq{a.cu, a.N, a.T, a.eq};
    const int cl = threadIdx.x % G, spb = BT / G, sl = threadIdx.x / G;
    const int c = ((int)blockIdx.y * G + cl) * V;
    if (c >= a.C) return;
    const int nv = a.C - c;
    const Taps<T, V, W> tp{(const T*)a.x + c, a.state ? (const T*)a.state + c : nullptr, a.xs, a.C, nv};

    if ((int)blockIdx.x >= strip_blocks) {  // the sequences' final states
        const int64_t rows = (int64_t)a.N * (W - 1);
        for (int64_t r = (int64_t)(blockIdx.x - strip_blocks) * spb + sl; r < rows;
             r += (int64_t)(gridDim.x - strip_blocks) * spb) {
            const int n = (int)(r / (W - 1)), i = (int)(r % (W - 1)), beg = sq.start(n);
            const int len = sq.start(n + 1) - beg;
            float v[V];
            tp.row(n, beg, (len > 0 ? len : 0) - (W - 1) + i, v);
            store_n<T, V>((T*)a.state_T + r * a.C + c, nv, v);
        }
        return;
    }

    const int tend = sq.end();
    int64_t t64 = ((int64_t)blockIdx.x * spb + sl) * L;
    if (t64 >= tend) return;
    int t = (int)t64;
    const int stop = (tend - t > L) ? t + L : tend;

    float w[V][W], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int ci = i < nv ? c + i : c;
#pragma unroll
        for (int j = 0; j < W; ++j) w[i][j] = a.weight[(int64_t)ci * W + j];
        b[i] = a.bias ? a.bias[ci] : 0.f;
    }
    int n = sq.find(t), beg = sq.start(n), end = sq.start(n + 1);
    float win[W - 1][V];  // rows t - W + 1 .. t - 1
#pragma unroll
    for (int k = 0; k < W - 1; ++k) tp.row(n, beg, t - beg - (W - 1) + k, win[k]);

    auto step = [&](int u, const float (&xv)[V]) {
        float z[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            z[i] = b[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) z[i] += w[i][j] * win[j][i];
            z[i] += w[i][W - 1] * xv[i];
            z[i] = act_f(z[i], a.silu);
#pragma unroll
            for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
            win[W - 2][i] = xv[i];
        }
        store_n<T, V>((T*)a.y + (int64_t)u * a.C + c, nv, z);
    };

    while (t < stop) {
        if (t + GRP <= stop && t + GRP <= end) {
            float xv[GRP][V];
#pragma unroll
            for (int i = 0; i < GRP; ++i) load_n<T, V>(tp.x + (int64_t)(t + i) * a.xs, nv, xv[i]);
#pragma unroll
            for (int i = 0; i < GRP; ++i) step(t + i, xv[i]);
            t += GRP;
        } else {
            const int until = stop - t > GRP ? t + GRP : stop;
#pragma unroll 1
            for (; t < until; ++t) {
                if (t >= end) {
                    n = sq.find(t);
                    beg = sq.start(n);
                    end = sq.start(n + 1);
                    if (end <= t) end = t + 1;  // offsets out of order: still one token at a time
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) tp.row(n, beg, t - beg - (W - 1) + k, win[k]);
                }
                float xv[V];
                load_n<T, V>(tp.x + (int64_t)t * a.xs, nv, xv);
                step(t, xv);
            }
        }
    }
}

// dz of token `pos` of sequence n (beg), from its taps
template <typename T, int V, int W>
__device__ __forceinline__ void dz_at(const ConvArgs& a, const Taps<T, V, W>& tp, const T* dyp, const float (&w)[V][W],
                                      const float (&b)[V], int n, int beg, int pos, float (&dz)[V]) {
    load_n<T, V>(dyp + (int64_t)(beg + pos) * a.ds, tp.n_valid, dz);
    if (!a.silu) return;
    float z[V];
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = b[i];
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float v[V];
        tp.row(n, beg, pos - (W - 1) + j, v);
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] += w[i][j] * v[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float s = sigmoid_f(z[i]);
        dz[i] *= s * (1.f + z[i] * (1.f - s));
    }
}

// Workgroups [0, strip_blocks) walk strips of tokens; the rest form the rows of
// dstate.  Both add the products x_s dz_{s+k} of the rows they own to their
// workgroup's partial dweight.
template <typename T, int V, int W>
__global__ __launch_bounds__(BT) void conv_bwd_kernel(ConvArgs a, int G, int L, int strip_blocks) {
    __shared__ float lds[BT * V];
    const Seqs sq{a.cu, a.N, a.T, a.eq};
    const int cl = threadIdx.x % G, spb = BT / G, sl = threadIdx.x / G;
    const int c0 = ((int)blockIdx.y * G + cl) * V;
    const bool live = c0 < a.C;  // idle lanes stay for the sums at the end
    const int c = live ? c0 : 0;
    const int nv = a.C - c;
    const Taps<T, V, W> tp{(const T*)a.x + c, a.state ? (const T*)a.state + c : nullptr, a.xs, a.C, nv};
    const T* dyp = (const T*)a.dy + c;

    float w[V][W], b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int ci = i < nv ? c + i : c;
#pragma unroll
        for (int j = 0; j < W; ++j) w[i][j] = a.weight[(int64_t)ci * W + j];
        b[i] = a.bias ? a.bias[ci] : 0.f;
    }
    float dw[W][V] = {}, db[V] = {};

    // row `pos` (state rows from -(W-1)) of sequence n by itself: its derivative
    // and its part of dw and db
    auto alone = [&](int n, int beg, int len, int pos, float (&dx)[V]) {
        float xv[V];
        tp.row(n, beg, pos, xv);
        if (pos >= len - (W - 1) && a.dstT) {
            load_n<T, V>((const T*)a.dstT + ((int64_t)n * (W - 1) + (pos - len + W - 1)) * a.C + c, nv, dx);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) dx[i] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const int p = pos + k;
            if (p < 0 || p >= len) continue;
            float dz[V];
            dz_at<T, V, W>(a, tp, dyp, w, b, n, beg, p, dz);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dx[i] += w[i][W - 1 - k] * dz[i];
                dw[W - 1 - k][i] += xv[i] * dz[i];
                if (k == 0) db[i] += dz[i];
            }
        }
    };

    if (live && (int)blockIdx.x >= strip_blocks) {
        const int64_t rows = (int64_t)a.N * (W - 1);
        for (int64_t r = (int64_t)(blockIdx.x - strip_blocks) * spb + sl; r < rows;
             r += (int64_t)(gridDim.x - strip_blocks) * spb) {
            const int n = (int)(r / (W - 1)), i = (int)(r % (W - 1)), beg = sq.start(n);
            int len = sq.start(n + 1) - beg;
            if (len < 0) len = 0;
            float dx[V];
            alone(n, beg, len, i - (W - 1), dx);
            if (a.state_T) store_n<T, V>((T*)a.state_T + r * a.C + c, nv, dx);
        }
    } else if (live) {
        const int tend = sq.end();
        const int64_t t64 = ((int64_t)blockIdx.x * spb + sl) * L;
        int t = t64 < tend ? (int)t64 : tend;
        const int stop = (tend - t > L) ? t + L : tend;
        int n = 0, beg = 0, end = 0;
        bool have = false;  // xw, dzw hold rows t .. t + W - 2
        float xw[W - 1][V], dzw[W - 1][V];
        while (t < stop) {
            if (t >= end) {
                n = sq.find(t);
                beg = sq.start(n);
                end = sq.start(n + 1);
                if (end <= t) end = t + 1;
                have = false;
            }
            if (t + GRP <= stop && t - (W - 1) >= beg && t + GRP + (W - 1) <= end) {
                if (!have) {
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) {
                        load_n<T, V>(tp.x + (int64_t)(t + k) * a.xs, nv, xw[k]);
                        dz_at<T, V, W>(a, tp, dyp, w, b, n, beg, t - beg + k, dzw[k]);
                    }
                    have = true;
                }
                float xv[GRP][V], dv[GRP][V];
#pragma unroll
                for (int i = 0; i < GRP; ++i) {
                    load_n<T, V>(tp.x + (int64_t)(t + W - 1 + i) * a.xs, nv, xv[i]);
                    load_n<T, V>(dyp + (int64_t)(t + W - 1 + i) * a.ds, nv, dv[i]);
                }
#pragma unroll
                for (int g = 0; g < GRP; ++g) {  // token t + g; the newest row is t + g + W - 1
                    float dx[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float dz = dv[g][i];
                        if (a.silu) {
                            float z = b[i];
#pragma unroll
                            for (int j = 0; j < W - 1; ++j) z += w[i][j] * xw[j][i];
                            z += w[i][W - 1] * xv[g][i];
                            const float s = sigmoid_f(z);
                            dz *= s * (1.f + z * (1.f - s));
                        }
                        float v = w[i][0] * dz;
                        dw[0][i] += xw[0][i] * dz;
#pragma unroll
                        for (int k = 0; k < W - 1; ++k) {
                            v += w[i][W - 1 - k] * dzw[k][i];
                            dw[W - 1 - k][i] += xw[0][i] * dzw[k][i];
                        }
                        db[i] += dzw[0][i];
                        dx[i] = v;
#pragma unroll
                        for (int k = 0; k < W - 2; ++k) {
                            xw[k][i] = xw[k + 1][i];
                            dzw[k][i] = dzw[k + 1][i];
                        }
                        xw[W - 2][i] = xv[g][i];
                        dzw[W - 2][i] = dz;
                    }
                    store_n<T, V>((T*)a.y + (int64_t)(t + g) * a.C + c, nv, dx);
                }
                t += GRP;
            } else {
                int until = stop - t > GRP ? t + GRP : stop;
                if (until > end) until = end;
                have = false;
#pragma unroll 1
                for (; t < until; ++t) {
                    float dx[V];
                    alone(n, beg, end - beg, t - beg, dx);
                    store_n<T, V>((T*)a.y + (int64_t)t * a.C + c, nv, dx);
                }
            }
        }
    }

    // the workgroup's partial sums, strip by strip in order
    float* out = a.part + (int64_t)blockIdx.x * a.C * (W + 1);
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) lds[threadIdx.x * V + i] = !live ? 0.f : j < W ? dw[j][i] : db[i];
        __syncthreads();
        if (sl == 0 && live) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float s = 0.f;
                for (int q = 0; q < spb; ++q) s += lds[(q * G + cl) * V + i];
                if (i < nv) out[j < W ? (int64_t)(c + i) * W + j : (int64_t)a.C * W + c + i] = s;
            }
        }
    }
}

// One token per sequence.
template <typename T, int V, int W>
__global__ __launch_bounds__(BT) void conv_step_kernel(ConvArgs a) {
    const int ncv = (a.C + V - 1) / V;
    const int64_t id = (int64_t)blockIdx.x * BT + threadIdx.x;
    if (id >= (int64_t)a.N * ncv) return;
    const int n = (int)(id / ncv), c = (int)(id % ncv) * V, nv = a.C - c;
    float win[W][V], z[V];
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        load_n<T, V>((const T*)a.state + ((int64_t)n * (W - 1) + k) * a.C + c, nv, win[k]);
    load_n<T, V>((const T*)a.x + (int64_t)n * a.xs + c, nv, win[W - 1]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int ci = i < nv ? c + i : c;
        z[i] = a.bias ? a.bias[ci] : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) z[i] += a.weight[(int64_t)ci * W + j] * win[j][i];
        z[i] = act_f(z[i], a.silu);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        store_n<T, V>((T*)a.state_T + ((int64_t)n * (W - 1) + k) * a.C + c, nv, win[k + 1]);
    store_n<T, V>((T*)a.y + (int64_t)n * a.C + c, nv, z);
}

// Lanes along the channels, strip length and strip workgroups.
struct ConvShape { int G, L, cblocks, strips; };
ConvShape conv_shape(int V, int T, int C, int max_blocks) {
    ConvShape s;
    const int ncv = (C + V - 1) / V;
    s.G = 64;
    while (s.G > 8 && s.G / 2 >= ncv) s.G /= 2;
    s.cblocks = (ncv + s.G - 1) / s.G;
    const int spb = BT / s.G;
    s.L = 8;
    while (s.L < 64 && ((int64_t)T + (int64_t)spb * s.L - 1) / ((int64_t)spb * s.L) * s.cblocks > 2048) s.L *= 2;
    // a bounded number of workgroups along the tokens (the backward's partial rows)
    while (max_blocks && ((int64_t)T + (int64_t)spb * s.L - 1) / ((int64_t)spb * s.L) > max_blocks) s.L *= 2;
    s.strips = (int)(((int64_t)T + (int64_t)spb * s.L - 1) / ((int64_t)spb * s.L));
    return s;
}

constexpr int BWD_STRIP_BLOCKS = 512;
int state_blocks(int N) { return N < 32 ? N : 32; }
int bwd_vec(int dtype) { return 4; }

#define KDA_CONV_RUN(KERNEL, T_, V_, GRID, ...)                                                                       \
    switch (a.W) {                                                                                                    \
        case 2: hipLaunchKernelGGL((KERNEL<T_, V_, 2>), GRID, dim3(BT), 0, st, __VA_ARGS__); break;                   \
        case 3: hipLaunchKernelGGL((KERNEL<T_, V_, 3>), GRID, dim3(BT), 0, st, __VA_ARGS__); break;                   \
        default: hipLaunchKernelGGL((KERNEL<T_, V_, 4>), GRID, dim3(BT), 0, st, __VA_ARGS__); break;                  \
    }

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t st) {
    const ConvShape s = conv_shape(a.dtype == 1 ? 8 : 4, a.T, a.C, 0);
    const int extra = a.state_T ? state_blocks(a.N) : 0;
    if (s.strips + extra == 0) return hipSuccess;
    const dim3 grid(s.strips + extra, s.cblocks);
    if (a.dtype == 1) { KDA_CONV_RUN(conv_fwd_kernel, bf16, 8, grid, a, s.G, s.L, s.strips) }
    else { KDA_CONV_RUN(conv_fwd_kernel, float, 4, grid, a, s.G, s.L, s.strips) }
    return hipGetLastError();
}

int conv_bwd_parts(int dtype, int T, int N, int C) {
    return conv_shape(bwd_vec(dtype), T, C, BWD_STRIP_BLOCKS).strips + state_blocks(N);
}

hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t st) {
    const ConvShape s = conv_shape(bwd_vec(a.dtype), a.T, a.C, BWD_STRIP_BLOCKS);
    const dim3 grid(s.strips + state_blocks(a.N), s.cblocks);
    if (a.dtype == 1) { KDA_CONV_RUN(conv_bwd_kernel, bf16, 4, grid, a, s.G, s.L, s.strips) }
    else { KDA_CONV_RUN(conv_bwd_kernel, float, 4, grid, a, s.G, s.L, s.strips) }
    return hipGetLastError();
}

hipError_t launch_conv_step(const ConvArgs& a, hipStream_t st) {
    const int V = a.dtype == 1 ? 8 : 4;
    const int64_t work = (int64_t)a.N * ((a.C + V - 1) / V);
    const dim3 grid((unsigned)((work + BT - 1) / BT));
    if (a.dtype == 1) { KDA_CONV_RUN(conv_step_kernel, bf16, 8, grid, a) }
    else { KDA_CONV_RUN(conv_step_kernel, float, 4, grid, a) }
    return hipGetLastError();
}

}  // namespace kda
