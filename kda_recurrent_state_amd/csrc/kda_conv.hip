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
// HBM-bound (forward 65501 x 4096 bf16: 5.8 TB/s; the backward, 4.9 TB/s, issues 29 vector
// instructions an element as well): a thread owns V adjacent channels of a strip of consecutive tokens
// and slides the W-token window along it in registers, so every row is read
// once and the strip's W - 1 leading rows (backward: 2 (W - 1)) once more,
// from cache.  Groups of tokens are loaded together ahead of their use.
// Groups that a sequence's edge crosses take a path of their own, which
// fetches each tap where the sequence says it is.
#include <type_traits>

#include "kda_block.hpp"
#include "kda_rows.hpp"

namespace kda {
namespace {

constexpr int BT = 256;
constexpr int GRP = 8, GRB = 4;  // tokens loaded together, forward and backward

template <bool SILU> __device__ __forceinline__ float act_f(float z) { return SILU ? z * sigmoid_f(z) : z; }

// One thread's view: V channels from c of the packed rows of x and the states.
template <typename T, int V, int W>
struct Taps {
    const T* x;
    const T* state;  // may be null
    const T* any;    // V readable elements, for a row that does not count
    int64_t xs;
    int C;
    uint32_t c;
    __device__ __forceinline__ Taps(const ConvArgs& a, int c_)
        : x((const T*)a.x), state((const T*)a.state), any((const T*)(a.weight + (int64_t)c_ * W)), xs(a.xs), C(a.C),
          c((uint32_t)c_) {}
    // row `pos` (from -(W-1)) of sequence n whose tokens start at beg, if it is
    // there; loaded either way, so that a caller's loads do not wait for each other
    __device__ __forceinline__ Pack<T, V> row(int n, int beg, int pos, bool there) const {
        const T* p = any;
        if (there && pos >= 0) p = x + (int64_t)(beg + pos) * xs + c;
        if (there && pos < 0 && state) p = state + ((int64_t)n * (W - 1) + (W - 1 + pos)) * C + c;
        return load_v<V>(p);
    }
    __device__ __forceinline__ bool counts(int pos) const { return pos >= 0 || state; }
};

template <int V, typename T>
__device__ __forceinline__ void get_if(bool there, const Pack<T, V>& r, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = there ? r[i] : 0.f;
}

// Taps and bias of V channels from c.
template <int V, int W>
__device__ __forceinline__ void load_weight(const ConvArgs& a, int c, float (&w)[V][W], float (&b)[V]) {
    const float* wp = a.weight + (int64_t)c * W;
    if constexpr (V * W % 4 != 0) {
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) w[i][j] = wp[i * W + j];
    } else {
        const Pack<float, V * W> wr = load_v<V * W>(wp);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) w[i][j] = wr[i * W + j];
    }
    if (a.bias) get_v<V>(load_v<V>(a.bias + c), b);
    else zero_v<V>(b);
}

// UNI: a strip is a whole wavefront's (G = 64), so its position and its rows'
// addresses stay in scalar registers and its sequence is found by all lanes.

// The sequence of token u, the first behind sequence n: the next one unless it is
// empty.
__device__ __forceinline__ void next_seq(const Seqs& sq, int u, int& n, int& beg, int& end) {
    if (n + 1 < sq.N && sq.start(n + 1) <= u && sq.start(n + 2) > u) n = n + 1;
    else n = sq.find(u);
    beg = sq.start(n);
    end = sq.start(n + 1);
    if (beg > u) beg = u;      // offsets out of order: still inside the tensors,
    if (end <= u) end = u + 1;  // and one token at a time
}

template <typename T, int V, int W, bool SILU, bool UNI, bool PAST>
__global__ __launch_bounds__(BT) void conv_fwd_kernel(ConvArgs a, int G, int L, int cblocks, int state_blocks) {
    const Seqs sq{a.cu, a.N, a.T, a.eq};
    const int cl = threadIdx.x % G, spb = BT / G;
    const int sl = UNI ? __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE) : threadIdx.x / G;
    // a token's columns by neighbouring workgroups, so that rows are read whole
    const int bx = (int)blockIdx.x / cblocks - state_blocks, at = ((int)blockIdx.x % cblocks * G + cl) * V;
    const int c = column<V>(at, a.C);
    const Taps<T, V, W> tp(a, c);

    if (bx < 0) {  // the sequences' final states
        const int64_t rows = (int64_t)a.N * (W - 1);
        for (int64_t r = (int64_t)(bx + state_blocks) * spb + sl; r < rows;
             r += (int64_t)state_blocks * spb) {
            const int n = (int)(r / (W - 1)), i = (int)(r % (W - 1)), beg = sq.start(n);
            const int len = sq.start(n + 1) - beg;
            const int pos = (len > 0 ? len : 0) - (W - 1) + i;
            float v[V];
            get_if<V>(tp.counts(pos), tp.row(n, beg, pos, true), v);
            if (at < a.C) store_v<V>((T*)a.state_T + r * a.C + c, v);
        }
        return;
    }

    const int tend = sq.end();
    const int64_t t64 = ((int64_t)bx * spb + sl) * L;
    if (t64 >= tend) return;
    int t = (int)t64;
    const int stop = (tend - t > L) ? t + L : tend;

    float w[V][W], b[V];
    load_weight<V, W>(a, c, w, b);
    int n = UNI ? wave_find(sq, t) : sq.find(t), beg = sq.start(n), end = sq.start(n + 1);
    if (beg > t) beg = t;  // (offsets out of order)
    if (at >= a.C) return;
    float win[W - 1][V];  // the rows before token u
    auto refill = [&](int u) {
        Pack<T, V> r[W - 1];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) r[k] = tp.row(n, beg, max(u - beg, 0) - (W - 1) + k, true);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) get_if<V>(tp.counts(u - beg - (W - 1) + k), r[k], win[k]);
    };
    refill(t);

    auto step = [&](int u, const Pack<T, V>& xr) {
        float z[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            z[i] = b[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) z[i] += w[i][j] * win[j][i];
            z[i] += w[i][W - 1] * xr[i];
            z[i] = act_f<SILU>(z[i]);
#pragma unroll
            for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
            win[W - 2][i] = xr[i];
        }
        store_nt<V>((T*)a.y + (int64_t)u * a.C + tp.c, z);
    };

    auto row = [&](int u) { return load_c<PAST, V>(tp.x + (int64_t)(u < a.T ? u : a.T - 1) * a.xs + tp.c); };
    while (t < stop) {
        if (t + GRP <= stop && t + GRP <= end) {
            Pack<T, V> xv[GRP];
#pragma unroll
            for (int i = 0; i < GRP; ++i) xv[i] = row(t + i);
#pragma unroll
            for (int i = 0; i < GRP; ++i) step(t + i, xv[i]);
            t += GRP;
        } else {
            const int until = stop - t > GRP ? t + GRP : stop;
            Pack<T, V> ahead = row(t);
#pragma unroll 1
            for (; t < until; ++t) {
                const Pack<T, V> xr = ahead;
                ahead = row(t + 1);
                if (t >= end) {
                    next_seq(sq, t, n, beg, end);
                    refill(t);
                }
                step(t, xr);
            }
        }
    }
}

// dy and z to dz
template <bool SILU> __device__ __forceinline__ float dz_of(float dy, float z) {
    if (!SILU) return dy;
    const float s = sigmoid_f(z);
    return dy * (s * (1.f + z * (1.f - s)));
}

// The first state_blocks rows of workgroups form the rows of dstate, the others
// walk strips of tokens.  Both add the products x_s dz_{s+k} of the rows they own to their
// workgroup's partial dweight.
template <typename T, int V, int W, bool SILU, bool UNI, bool PAST>
__global__ __launch_bounds__(BT) void conv_bwd_kernel(ConvArgs a, int G, int L, int cblocks, int state_blocks) {
    __shared__ float lds[BT * V];
    const Seqs sq{a.cu, a.N, a.T, a.eq};
    const int cl = threadIdx.x % G, spb = BT / G;
    const int sl = UNI ? __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE) : threadIdx.x / G;
    const int bx = (int)blockIdx.x / cblocks - state_blocks, c0 = ((int)blockIdx.x % cblocks * G + cl) * V;
    const bool live = c0 < a.C;  // idle lanes stay for the sums at the end
    const int c = column<V>(c0, a.C);
    const Taps<T, V, W> tp(a, c);
    const T* dyp = (const T*)a.dy;

    float w[V][W], b[V];
    load_weight<V, W>(a, c, w, b);
    float dw[W][V] = {}, db[V] = {};

    // row `pos` (state rows from -(W-1)) of sequence n by itself: its derivative
    // and its part of dw and db
    auto alone = [&](int n, int beg, int len, int pos, float (&dx)[V]) {
        Pack<T, V> xr[2 * W - 1], dr[W];
#pragma unroll
        for (int k = 0; k < 2 * W - 1; ++k) {
            const int q = pos - (W - 1) + k;
            xr[k] = tp.row(n, beg, q, q >= -(W - 1) && q < len);
        }
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const int q = pos + k;
            dr[k] = load_v<V>(q >= 0 && q < len ? dyp + (int64_t)(beg + q) * a.ds + tp.c : tp.any);
        }
        const bool out = pos >= len - (W - 1) && a.dstT;  // the row is one of the outgoing state's
        const Pack<T, V> sr =
            load_v<V>(out ? (const T*)a.dstT + ((int64_t)n * (W - 1) + (pos - len + W - 1)) * a.C + c : tp.any);
        get_if<V>(out, sr, dx);
        float xf[2 * W - 1][V];
#pragma unroll
        for (int k = 0; k < 2 * W - 1; ++k) {
            const int q = pos - (W - 1) + k;
            get_if<V>(q >= -(W - 1) && q < len && tp.counts(q), xr[k], xf[k]);
        }
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const bool there = pos + k >= 0 && pos + k < len;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float z = b[i];
#pragma unroll
                for (int j = 0; j < W; ++j) z += w[i][j] * xf[k + j][i];
                const float dz = there ? dz_of<SILU>(dr[k][i], z) : 0.f;
                dx[i] += w[i][W - 1 - k] * dz;
                dw[W - 1 - k][i] += there ? xf[W - 1][i] * dz : 0.f;
                if (k == 0) db[i] += dz;
            }
        }
    };

    if (live && bx < 0) {
        const int64_t rows = (int64_t)a.N * (W - 1);
        for (int64_t r = (int64_t)(bx + state_blocks) * spb + sl; r < rows;
             r += (int64_t)state_blocks * spb) {
            const int n = (int)(r / (W - 1)), i = (int)(r % (W - 1)), beg = sq.start(n);
            int len = sq.start(n + 1) - beg;
            if (len < 0) len = 0;
            float dx[V];
            alone(n, beg, len, i - (W - 1), dx);
            if (a.state_T) store_v<V>((T*)a.state_T + r * a.C + tp.c, dx);
        }
    } else if (live) {
        const int tend = sq.end();
        const int64_t t64 = ((int64_t)bx * spb + sl) * L;
        int t = t64 < tend ? (int)t64 : tend;
        const int stop = (tend - t > L) ? t + L : tend;
        int n = 0, beg = 0, end = 0;
        if (UNI && t < stop && !~__ballot(1)) {  // all lanes are here
            n = wave_find(sq, t);
            beg = min(sq.start(n), t);
            end = max(sq.start(n + 1), t + 1);
        }
        bool have = false;  // xw, dzw hold rows t .. t + W - 2
        float xw[W - 1][V], dzw[W - 1][V];
        while (t < stop) {
            if (t >= end) {
                next_seq(sq, t, n, beg, end);
                have = false;
            }
            if (t + GRB <= stop && t - (W - 1) >= beg && t + GRB + (W - 1) <= end) {
                if (!have) {
                    Pack<T, V> r[2 * (W - 1)], d[W - 1];  // x rows from t - W + 1, dy rows from t
#pragma unroll
                    for (int k = 0; k < 2 * (W - 1); ++k)
                        r[k] = load_v<V>(tp.x + (int64_t)(t - (W - 1) + k) * a.xs + tp.c);
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) d[k] = load_v<V>(dyp + (int64_t)(t + k) * a.ds + tp.c);
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) {
                        get_v<V>(r[W - 1 + k], xw[k]);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            float z = b[i];
#pragma unroll
                            for (int j = 0; j < W; ++j) z += w[i][j] * r[k + j][i];
                            dzw[k][i] = dz_of<SILU>(d[k][i], z);
                        }
                    }
                    have = true;
                }
                Pack<T, V> xv[GRB], dv[GRB];
#pragma unroll
                for (int i = 0; i < GRB; ++i) {
                    xv[i] = load_c<PAST, V>(tp.x + (int64_t)(t + W - 1 + i) * a.xs + tp.c);
                    dv[i] = load_c<PAST, V>(dyp + (int64_t)(t + W - 1 + i) * a.ds + tp.c);
                }
#pragma unroll
                for (int g = 0; g < GRB; ++g) {  // token t + g; the newest row is t + g + W - 1
                    float dx[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float z = b[i];
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) z += w[i][j] * xw[j][i];
                        z += w[i][W - 1] * xv[g][i];
                        const float dz = dz_of<SILU>(dv[g][i], z);
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
                    store_nt<V>((T*)a.y + (int64_t)(t + g) * a.C + tp.c, dx);
                }
                t += GRB;
            } else {
                int until = stop - t > GRB ? t + GRB : stop;
                if (until > end) until = end;
                have = false;
#pragma unroll 1
                for (; t < until; ++t) {
                    float dx[V];
                    alone(n, beg, end - beg, t - beg, dx);
                    store_v<V>((T*)a.y + (int64_t)t * a.C + tp.c, dx);
                }
            }
        }
    }

    // the workgroup's partial sums, strip by strip in order
    float* out = a.part + (int64_t)(bx + state_blocks) * a.C * (W + 1);
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
                out[j < W ? (int64_t)(c + i) * W + j : (int64_t)a.C * W + c + i] = s;
            }
        }
    }
}

// One token per sequence.  The state may be updated in place, so a lane owns its
// columns alone: the row's last few go one by one (a vector at the row's end that
// overlapped its neighbour's could read what that lane has already written).
template <typename T, int V, int W, bool SILU>
__device__ __forceinline__ void conv_step_at(const ConvArgs& a, int n, int c) {
    const T* st = (const T*)a.state + (int64_t)n * (W - 1) * a.C + c;
    Pack<T, V> r[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) r[k] = load_v<V>(st + (int64_t)k * a.C);
    r[W - 1] = load_v<V>((const T*)a.x + (int64_t)n * a.xs + c);
    float w[V][W], z[V];
    load_weight<V, W>(a, c, w, z);
    T* to = (T*)a.state_T + (int64_t)n * (W - 1) * a.C + c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int j = 0; j < W; ++j) z[i] += w[i][j] * r[j][i];
        z[i] = act_f<SILU>(z[i]);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) *reinterpret_cast<Pack<T, V>*>(to + (int64_t)k * a.C) = r[k + 1];
    store_v<V>((T*)a.y + (int64_t)n * a.C + c, z);
}

template <typename T, int V, int W, bool SILU>
__global__ __launch_bounds__(BT) void conv_step_kernel(ConvArgs a) {
    const int ncv = (a.C + V - 1) / V;
    const int64_t id = (int64_t)blockIdx.x * BT + threadIdx.x;
    if (id >= (int64_t)a.N * ncv) return;
    const int n = (int)(id / ncv), c = (int)(id % ncv) * V;
    if (c + V <= a.C) {
        conv_step_at<T, V, W, SILU>(a, n, c);
    } else {
        for (int i = c; i < a.C; ++i) conv_step_at<T, 1, W, SILU>(a, n, i);
    }
}

// Lanes along the channels, strip length and strip workgroups.
struct ConvShape { int G, L, cblocks, strips; };
ConvShape conv_shape(int V, int C) {
    ConvShape s;
    const int ncv = (C + V - 1) / V;
    s.G = 64;  // fewer in narrow rows (65536 x 64: 11 us with 8 lanes a row, 20 with 64)
    while (s.G > 8 && s.G / 2 >= ncv) s.G /= 2;
    s.cblocks = (ncv + s.G - 1) / s.G;
    s.L = s.strips = 0;
    return s;
}
void set_strips(ConvShape* s, int T, int64_t L) {
    const int64_t spb = BT / s->G;
    s->L = (int)L;
    s->strips = (int)((T + spb * L - 1) / (spb * L));
}
// Forward: strips of 16 tokens (65501 x 4096 bf16: 185 us; 8: 194, 32: 189, 64: 199), or
// of 8 where those make no more than 2048 workgroups.
ConvShape fwd_shape(int V, int T, int C) {
    ConvShape s = conv_shape(V, C);
    int L = 8;
    const int64_t spb = BT / s.G;
    while (L < 16 && (T + spb * L - 1) / (spb * L) * s.cblocks > 2048) L *= 2;
    set_strips(&s, T, L);
    return s;
}
// Backward: strips of one length that fill the GPU (1024 workgroups, four per
// compute unit) in as many whole rounds as keep them near 128 tokens; at most
// 512 along the tokens, each of which leaves a partial row.
ConvShape bwd_shape(int V, int T, int C) {
    ConvShape s = conv_shape(V, C);
    const int64_t spb = BT / s.G, fill = spb * 1024;
    const int64_t one = ((int64_t)T * s.cblocks + fill - 1) / fill, rounds = (one + 127) / 128;
    int64_t L = one == 0 ? 1 : (one + rounds - 1) / rounds;
    const int64_t least = (T + spb * 512 - 1) / (spb * 512);
    if (L < least) L = least;
    if (L < 2 * GRB) L = 2 * GRB;
    set_strips(&s, T, (L + GRB - 1) / GRB * GRB);
    return s;
}

int state_blocks(int N) { return N < 32 ? N : 32; }
// Channels per lane.  Forward: 16 bytes (65501 x 4096 bf16: 185 us; four channels 192).
// Backward: 2, whose windows and sums leave more wavefronts than 4 (30000 x 1536 with
// three taps: 72 us against 78; 3000 x 1024 with four: 20 against 24; 32768 x 4096: 170
// against 169; fp32, 20011 x 2000: 118 against 115).  Single channels in rows shorter than that.
int fwd_vec(int dtype, int C) { return dtype == 1 ? (C >= 8 ? 8 : 1) : (C >= 4 ? 4 : 1); }
int bwd_vec(int C) { return C >= 2 ? 2 : 1; }

// f(taps, SiLU or not) for the call's.
template <typename F> void by_taps(const ConvArgs& a, F f) {
    auto act = [&](auto w) {
        if (a.silu) f(w, std::true_type{});
        else f(w, std::false_type{});
    };
    if (a.W == 2) act(std::integral_constant<int, 2>{});
    else if (a.W == 3) act(std::integral_constant<int, 3>{});
    else act(std::integral_constant<int, 4>{});
}

// The grid of rows x cblocks workgroups; a launch has fewer than 2^32 threads.
bool grid_of(const ConvShape& s, int extra, dim3* grid) {
    const int64_t blocks = ((int64_t)s.strips + extra) * s.cblocks;
    *grid = dim3((unsigned)blocks);
    return blocks <= 0xffffffffll / BT;
}

#define KDA_CONV_LAUNCH(KERNEL, ...) \
    hipLaunchKernelGGL((KERNEL<T, V, W, SILU, __VA_ARGS__>), grid, dim3(BT), 0, st, a, s.G, s.L, s.cblocks, extra)
#define KDA_CONV_CASES(KERNEL, PAST)                                           \
    by_taps(a, [&](auto w, auto silu) {                                        \
        constexpr int W = decltype(w)::value;                                  \
        constexpr bool SILU = decltype(silu)::value, WIDE = V > 1;             \
        if (!WIDE || s.G < WAVE) KDA_CONV_LAUNCH(KERNEL, false, false);        \
        else if (PAST) KDA_CONV_LAUNCH(KERNEL, WIDE, WIDE);                    \
        else KDA_CONV_LAUNCH(KERNEL, WIDE, false);                             \
    })
template <typename T, int V> hipError_t fwd_launch(const ConvArgs& a, hipStream_t st) {
    const ConvShape s = fwd_shape(V, a.T, a.C);
    const int extra = a.state_T ? state_blocks(a.N) : 0;
    const int64_t size = (int64_t)a.T * a.C * sizeof(T);
    dim3 grid;
    if (!grid_of(s, extra, &grid)) return hipErrorInvalidConfiguration;
    if (grid.x == 0) return hipSuccess;
    KDA_CONV_CASES(conv_fwd_kernel, past_cache(size));
    return hipGetLastError();
}

template <typename T, int V> hipError_t bwd_launch(const ConvArgs& a, hipStream_t st) {
    const ConvShape s = bwd_shape(V, a.T, a.C);
    const int extra = state_blocks(a.N);
    const int64_t size = (int64_t)a.T * a.C * sizeof(T);
    dim3 grid;
    if (!grid_of(s, extra, &grid)) return hipErrorInvalidConfiguration;
    KDA_CONV_CASES(conv_bwd_kernel, past_cache(2 * size));
    return hipGetLastError();
}

template <typename T, int V> hipError_t step_launch(const ConvArgs& a, hipStream_t st) {
    const int64_t work = (int64_t)a.N * ((a.C + V - 1) / V);
    by_taps(a, [&](auto w, auto silu) {
        hipLaunchKernelGGL((conv_step_kernel<T, V, decltype(w)::value, decltype(silu)::value>),
                           dim3((unsigned)((work + BT - 1) / BT)), dim3(BT), 0, st, a);
    });
    return hipGetLastError();
}

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t st) {
    const int v = fwd_vec(a.dtype, a.C);
    if (a.dtype == 1) return v == 1 ? fwd_launch<bf16, 1>(a, st) : fwd_launch<bf16, 8>(a, st);
    return v == 1 ? fwd_launch<float, 1>(a, st) : fwd_launch<float, 4>(a, st);
}

int conv_bwd_parts(int T, int N, int C) { return bwd_shape(bwd_vec(C), T, C).strips + state_blocks(N); }

hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t st) {
    const int v = bwd_vec(a.C);
    if (a.dtype == 1) return v == 1 ? bwd_launch<bf16, 1>(a, st) : bwd_launch<bf16, 2>(a, st);
    return v == 1 ? bwd_launch<float, 1>(a, st) : bwd_launch<float, 2>(a, st);
}

hipError_t launch_conv_step(const ConvArgs& a, hipStream_t st) {
    const int v = fwd_vec(a.dtype, a.C);
    if (a.dtype == 1) return v == 1 ? step_launch<bf16, 1>(a, st) : step_launch<bf16, 8>(a, st);
    return v == 1 ? step_launch<float, 1>(a, st) : step_launch<float, 4>(a, st);
}

}  // namespace kda
