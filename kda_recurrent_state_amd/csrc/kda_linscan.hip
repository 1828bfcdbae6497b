// kda_linscan.hip -- diagonal gated linear recurrence over packed sequences on gfx950.
//
//   h_t = a_t h_{t-1} + x_t,  a_t = e^{log a_t},  y_t = h_t            per channel
//   g_t = dy_t + a_{t+1} g_{t+1},  dx_t = g_t,  dlog a_t = g_t a_t h_{t-1}
//
// The packed axis is cut into tiles of 64 tokens whatever the sequences'
// edges; a workgroup holds one tile of 64 V channels, each of its four
// wavefronts 16 tokens in registers.  A run of tokens maps the state before it
// to P h + E (P the product of its a, E its end from a zero state), or, if a
// sequence starts in it, to E alone: that case is marked by P = -1 and chosen,
// never multiplied, so that nothing of an earlier sequence, infinities
// included, reaches the next one.  The backward runs the same way from the
// end, with c_t = a_t g_t as what a token hands to the one before it.
#include "kda_block.hpp"
#include "kda_rows.hpp"

namespace kda {
namespace {

constexpr int TT = LINSCAN_TILE;      // tokens per tile
constexpr int NW = 4, BT = NW * WAVE;  // wavefronts of a workgroup
constexpr int TW = TT / NW;           // tokens per wavefront

// One run of tokens followed by another: (p, e) <- (p2, e2) after (p, e).
__device__ __forceinline__ void then(float& p, float& e, float p2, float e2) {
    e = p2 < 0.f ? e2 : p2 * e + e2;
    p = p2 < 0.f ? -1.f : p < 0.f ? -1.f : p2 * p;
}
__device__ __forceinline__ float apply(float p, float e, float h) { return p < 0.f ? e : p * h + e; }

// Which of a wavefront's tokens start and end a sequence (uniform over the
// wavefront): bit i of first / last for token t0 + i.
struct Edges {
    uint32_t first, last;
    int count;  // tokens of the run that exist
};
__device__ __forceinline__ Edges edges_of(const Seqs& sq, int t0, int tend) {
    Edges e{0u, 0u, tend - t0 < TW ? tend - t0 : TW};
    if (e.count <= 0) { e.count = 0; return e; }
    int t = t0;
    while (t < t0 + e.count) {
        const int n = sq.find(t);
        if (sq.start(n) == t) e.first |= 1u << (t - t0);
        int nx = sq.start(n + 1);
        if (nx <= t) nx = t + 1;
        if (nx <= t0 + e.count) e.last |= 1u << (nx - 1 - t0);
        t = nx;
    }
    return e;
}

// a and x of a wavefront's tokens; absent tokens are the identity.
template <typename T, int V>
__device__ __forceinline__ void load_run(const LinScanArgs& p, int t0, int count, int c, int nv, float (&a)[TW][V],
                                         float (&x)[TW][V]) {
#pragma unroll
    for (int i = 0; i < TW; ++i) {
        if (i < count) {
            load_n<float, V>(p.la + (int64_t)(t0 + i) * p.ls + c, nv, a[i]);
            load_n<T, V>((const T*)p.x + (int64_t)(t0 + i) * p.xs + c, nv, x[i]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) a[i][v] = x[i][v] = 0.f;
        }
    }
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) a[i][v] = __expf(a[i][v]);
}

template <int V>
__device__ __forceinline__ void load_h0(const LinScanArgs& p, const float* h0, int n, int c, int nv, float (&h)[V]) {
    if (h0) {
        load_n<float, V>(h0 + (int64_t)n * p.C + c, nv, h);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = 0.f;
    }
}

// (P, E) of a wavefront's run, forwards
template <int V>
__device__ __forceinline__ void run_forward(const LinScanArgs& p, const Seqs& sq, const Edges& ed, int t0, int c, int nv,
                                            const float (&a)[TW][V], const float (&x)[TW][V], float (&P)[V],
                                            float (&E)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.f, E[v] = 0.f;
#pragma unroll
    for (int i = 0; i < TW; ++i) {
        if (ed.first >> i & 1) {
            load_h0<V>(p, p.h0, sq.find(t0 + i), c, nv, E);
#pragma unroll
            for (int v = 0; v < V; ++v) P[v] = -1.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            E[v] = a[i][v] * E[v] + x[i][v];
            P[v] = P[v] < 0.f ? -1.f : P[v] * a[i][v];
        }
    }
}

// (P, E) of every tile: agg[tile][0][c] = P, agg[tile][1][c] = E
template <typename T, int V>
__global__ __launch_bounds__(BT) void linscan_agg_kernel(LinScanArgs p) {
    __shared__ float sp[NW][WAVE * V], se[NW][WAVE * V];
    const Seqs sq{p.cu, p.N, p.T, p.eq};
    const int lane = threadIdx.x % WAVE, wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int c = ((int)blockIdx.y * WAVE + lane) * V, nv = p.C - c;
    const int t0 = (int)blockIdx.x * TT + wv * TW;
    const Edges ed = edges_of(sq, t0, sq.end());
    float a[TW][V], x[TW][V], P[V], E[V];
    load_run<T, V>(p, t0, ed.count, c, nv, a, x);
    run_forward<V>(p, sq, ed, t0, c, nv, a, x, P, E);
#pragma unroll
    for (int v = 0; v < V; ++v) sp[wv][lane * V + v] = P[v], se[wv][lane * V + v] = E[v];
    __syncthreads();
    if (wv == 0) {
#pragma unroll
        for (int w = 1; w < NW; ++w)
#pragma unroll
            for (int v = 0; v < V; ++v) then(P[v], E[v], sp[w][lane * V + v], se[w][lane * V + v]);
        store_n<float, V>(p.agg + (int64_t)blockIdx.x * 2 * p.C + c, nv, P);
        store_n<float, V>(p.agg + ((int64_t)blockIdx.x * 2 + 1) * p.C + c, nv, E);
    }
}

// The same from the end: what a tile hands to the token before it, P c + E for
// c handed to it from behind.  Absent tokens are the identity.
template <typename T, int V>
__device__ __forceinline__ void run_backward(const LinScanArgs& p, const Seqs& sq, const Edges& ed, int t0, int c,
                                             int nv, const float (&a)[TW][V], const float (&dy)[TW][V], float (&P)[V],
                                             float (&E)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.f, E[v] = 0.f;
#pragma unroll
    for (int i = TW - 1; i >= 0; --i) {
        if (i >= ed.count) continue;
        if (ed.last >> i & 1) {
            load_h0<V>(p, p.dhT, sq.find(t0 + i), c, nv, E);
#pragma unroll
            for (int v = 0; v < V; ++v) P[v] = -1.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            E[v] = a[i][v] * (dy[i][v] + E[v]);
            P[v] = P[v] < 0.f ? -1.f : P[v] * a[i][v];
        }
    }
}

template <typename T, int V>
__global__ __launch_bounds__(BT) void linscan_ragg_kernel(LinScanArgs p) {
    __shared__ float sp[NW][WAVE * V], se[NW][WAVE * V];
    const Seqs sq{p.cu, p.N, p.T, p.eq};
    const int lane = threadIdx.x % WAVE, wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int c = ((int)blockIdx.y * WAVE + lane) * V, nv = p.C - c;
    const int t0 = (int)blockIdx.x * TT + wv * TW;
    const Edges ed = edges_of(sq, t0, sq.end());
    LinScanArgs q = p;
    q.x = p.dy;
    q.xs = p.ds;
    float a[TW][V], dy[TW][V], P[V], E[V];
    load_run<T, V>(q, t0, ed.count, c, nv, a, dy);
    run_backward<T, V>(p, sq, ed, t0, c, nv, a, dy, P, E);
#pragma unroll
    for (int v = 0; v < V; ++v) sp[wv][lane * V + v] = P[v], se[wv][lane * V + v] = E[v];
    __syncthreads();
    if (wv == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) P[v] = sp[NW - 1][lane * V + v], E[v] = se[NW - 1][lane * V + v];
#pragma unroll
        for (int w = NW - 2; w >= 0; --w)
#pragma unroll
            for (int v = 0; v < V; ++v) then(P[v], E[v], sp[w][lane * V + v], se[w][lane * V + v]);
        store_n<float, V>(p.agg + (int64_t)blockIdx.x * 2 * p.C + c, nv, P);
        store_n<float, V>(p.agg + ((int64_t)blockIdx.x * 2 + 1) * p.C + c, nv, E);
    }
}

// Carries between tiles, one thread per channel: carry[tile] = the state before
// (reverse: handed from behind to) the tile.
constexpr int CB = 16;  // tiles read ahead
__global__ __launch_bounds__(WAVE) void linscan_carry_kernel(const float* agg, float* carry, int tiles, int C,
                                                             int reverse) {
    const int c = (int)blockIdx.x * WAVE + threadIdx.x;
    if (c >= C) return;
    float h = 0.f;
    for (int k0 = 0; k0 < tiles; k0 += CB) {
        float P[CB], E[CB];
#pragma unroll
        for (int i = 0; i < CB; ++i) {
            const int k = k0 + i < tiles ? k0 + i : tiles - 1;
            const int64_t tile = reverse ? tiles - 1 - k : k;
            P[i] = agg[tile * 2 * C + c];
            E[i] = agg[(tile * 2 + 1) * C + c];
        }
#pragma unroll
        for (int i = 0; i < CB; ++i) {
            if (k0 + i < tiles) {
                const int64_t tile = reverse ? tiles - 1 - (k0 + i) : k0 + i;
                carry[tile * C + c] = h;
                h = apply(P[i], E[i], h);
            }
        }
    }
}

// The last workgroups of the output kernels: an empty sequence's final state is
// its initial one (forward: hT from h0, backward: dh0 from dhT).
__device__ __forceinline__ void empty_seqs(const Seqs& sq, const float* from, float* to, int C, int block, int blocks) {
    for (int n = block; n < sq.N; n += blocks) {
        if (sq.start(n + 1) > sq.start(n)) continue;
        for (int c = threadIdx.x; c < C; c += BT) to[(int64_t)n * C + c] = from ? from[(int64_t)n * C + c] : 0.f;
    }
}

template <typename T, int V>
__global__ __launch_bounds__(BT) void linscan_fwd_kernel(LinScanArgs p, int tiles) {
    __shared__ float sp[NW][WAVE * V], se[NW][WAVE * V];
    const Seqs sq{p.cu, p.N, p.T, p.eq};
    if ((int)blockIdx.x >= tiles) {
        if (blockIdx.y == 0) empty_seqs(sq, p.h0, p.hT, p.C, blockIdx.x - tiles, gridDim.x - tiles);
        return;
    }
    const int lane = threadIdx.x % WAVE, wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int c = ((int)blockIdx.y * WAVE + lane) * V, nv = p.C - c;
    const int t0 = (int)blockIdx.x * TT + wv * TW;
    const Edges ed = edges_of(sq, t0, sq.end());
    float a[TW][V], x[TW][V], P[V], E[V], h[V];
    load_n<float, V>(p.states + (int64_t)blockIdx.x * p.C + c, nv, h);
    load_run<T, V>(p, t0, ed.count, c, nv, a, x);
    run_forward<V>(p, sq, ed, t0, c, nv, a, x, P, E);
#pragma unroll
    for (int v = 0; v < V; ++v) sp[wv][lane * V + v] = P[v], se[wv][lane * V + v] = E[v];
    __syncthreads();
    for (int w = 0; w < wv; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = apply(sp[w][lane * V + v], se[w][lane * V + v], h[v]);
#pragma unroll
    for (int i = 0; i < TW; ++i) {
        if (i >= ed.count) continue;
        if (ed.first >> i & 1) load_h0<V>(p, p.h0, sq.find(t0 + i), c, nv, h);
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = a[i][v] * h[v] + x[i][v];
        store_n<T, V>((T*)p.y + (int64_t)(t0 + i) * p.C + c, nv, h);
        if ((ed.last >> i & 1) && p.hT) store_n<float, V>(p.hT + (int64_t)sq.find(t0 + i) * p.C + c, nv, h);
    }
}

template <typename T, int V>
__global__ __launch_bounds__(BT) void linscan_bwd_kernel(LinScanArgs p, int tiles) {
    __shared__ float sp[NW][WAVE * V], se[NW][WAVE * V], rp[NW][WAVE * V], re[NW][WAVE * V];
    const Seqs sq{p.cu, p.N, p.T, p.eq};
    if ((int)blockIdx.x >= tiles) {
        if (blockIdx.y == 0) empty_seqs(sq, p.dhT, p.hT, p.C, blockIdx.x - tiles, gridDim.x - tiles);
        return;
    }
    const int lane = threadIdx.x % WAVE, wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int c = ((int)blockIdx.y * WAVE + lane) * V, nv = p.C - c;
    const int t0 = (int)blockIdx.x * TT + wv * TW;
    const Edges ed = edges_of(sq, t0, sq.end());
    float a[TW][V], x[TW][V], dy[TW][V], P[V], E[V], h[V], g[V];
    load_n<float, V>(p.states + (int64_t)blockIdx.x * p.C + c, nv, h);
    load_n<float, V>(p.rcarry + (int64_t)blockIdx.x * p.C + c, nv, g);
    load_run<T, V>(p, t0, ed.count, c, nv, a, x);
#pragma unroll
    for (int i = 0; i < TW; ++i) {
        if (i < ed.count) load_n<T, V>((const T*)p.dy + (int64_t)(t0 + i) * p.ds + c, nv, dy[i]);
    }
    run_forward<V>(p, sq, ed, t0, c, nv, a, x, P, E);
#pragma unroll
    for (int v = 0; v < V; ++v) sp[wv][lane * V + v] = P[v], se[wv][lane * V + v] = E[v];
    run_backward<T, V>(p, sq, ed, t0, c, nv, a, dy, P, E);
#pragma unroll
    for (int v = 0; v < V; ++v) rp[wv][lane * V + v] = P[v], re[wv][lane * V + v] = E[v];
    __syncthreads();
    for (int w = 0; w < wv; ++w)
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = apply(sp[w][lane * V + v], se[w][lane * V + v], h[v]);
    for (int w = NW - 1; w > wv; --w)
#pragma unroll
        for (int v = 0; v < V; ++v) g[v] = apply(rp[w][lane * V + v], re[w][lane * V + v], g[v]);
    // x[i] becomes the state before token i
#pragma unroll
    for (int i = 0; i < TW; ++i) {
        if (ed.first >> i & 1) load_h0<V>(p, p.h0, sq.find(t0 + i), c, nv, h);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float xi = x[i][v];
            x[i][v] = h[v];
            h[v] = a[i][v] * h[v] + xi;
        }
    }
#pragma unroll
    for (int i = TW - 1; i >= 0; --i) {
        if (i >= ed.count) continue;
        if (ed.last >> i & 1) load_h0<V>(p, p.dhT, sq.find(t0 + i), c, nv, g);
        float dl[V];
#pragma unroll
        for (int v = 0; v < V; ++v) dy[i][v] += g[v];
        store_n<T, V>((T*)p.y + (int64_t)(t0 + i) * p.C + c, nv, dy[i]);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            g[v] = a[i][v] * dy[i][v];
            dl[v] = g[v] * x[i][v];
        }
        store_n<float, V>(p.dla + (int64_t)(t0 + i) * p.C + c, nv, dl);
        if ((ed.first >> i & 1) && p.hT) store_n<float, V>(p.hT + (int64_t)sq.find(t0 + i) * p.C + c, nv, g);
    }
}

template <typename T, int V>
__global__ __launch_bounds__(BT) void linscan_step_kernel(LinScanArgs p) {
    const int ncv = (p.C + V - 1) / V;
    const int64_t id = (int64_t)blockIdx.x * BT + threadIdx.x;
    if (id >= (int64_t)p.N * ncv) return;
    const int n = (int)(id / ncv), c = (int)(id % ncv) * V, nv = p.C - c;
    float a[V], x[V], h[V];
    load_n<float, V>(p.la + (int64_t)n * p.ls + c, nv, a);
    load_n<T, V>((const T*)p.x + (int64_t)n * p.xs + c, nv, x);
    load_n<float, V>(p.h0 + (int64_t)n * p.C + c, nv, h);
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = __expf(a[v]) * h[v] + x[v];
    store_n<float, V>(p.hT + (int64_t)n * p.C + c, nv, h);
    store_n<T, V>((T*)p.y + (int64_t)n * p.C + c, nv, h);
}

int tiles_of(int T) { return (T + TT - 1) / TT; }
dim3 tile_grid(int tiles, int C, int V) { return dim3(tiles, (C + WAVE * V - 1) / (WAVE * V)); }
int empty_blocks(int N) { return N < 64 ? N : 64; }
constexpr int VF = 4, VB = 2;  // channels per lane, forward and backward

}  // namespace

hipError_t launch_linscan_states(const LinScanArgs& a, hipStream_t st) {
    const int tiles = tiles_of(a.T);
    if (a.dtype == 1) hipLaunchKernelGGL((linscan_agg_kernel<bf16, VF>), tile_grid(tiles, a.C, VF), dim3(BT), 0, st, a);
    else hipLaunchKernelGGL((linscan_agg_kernel<float, VF>), tile_grid(tiles, a.C, VF), dim3(BT), 0, st, a);
    hipLaunchKernelGGL(linscan_carry_kernel, dim3((a.C + WAVE - 1) / WAVE), dim3(WAVE), 0, st, a.agg, a.states, tiles,
                       a.C, 0);
    return hipGetLastError();
}

hipError_t launch_linscan_fwd(const LinScanArgs& a, hipStream_t st) {
    const int tiles = tiles_of(a.T);
    dim3 grid = tile_grid(tiles, a.C, VF);
    grid.x += a.hT ? empty_blocks(a.N) : 0;
    if (grid.x == 0) return hipSuccess;
    if (a.dtype == 1) hipLaunchKernelGGL((linscan_fwd_kernel<bf16, VF>), grid, dim3(BT), 0, st, a, tiles);
    else hipLaunchKernelGGL((linscan_fwd_kernel<float, VF>), grid, dim3(BT), 0, st, a, tiles);
    return hipGetLastError();
}

hipError_t launch_linscan_bwd(const LinScanArgs& a, hipStream_t st) {
    const int tiles = tiles_of(a.T);
    if (tiles > 0) {
        if (a.dtype == 1)
            hipLaunchKernelGGL((linscan_ragg_kernel<bf16, VF>), tile_grid(tiles, a.C, VF), dim3(BT), 0, st, a);
        else
            hipLaunchKernelGGL((linscan_ragg_kernel<float, VF>), tile_grid(tiles, a.C, VF), dim3(BT), 0, st, a);
        hipLaunchKernelGGL(linscan_carry_kernel, dim3((a.C + WAVE - 1) / WAVE), dim3(WAVE), 0, st, a.agg, a.rcarry,
                           tiles, a.C, 1);
    }
    dim3 grid = tile_grid(tiles, a.C, VB);
    grid.x += a.hT ? empty_blocks(a.N) : 0;
    if (grid.x == 0) return hipSuccess;
    if (a.dtype == 1) hipLaunchKernelGGL((linscan_bwd_kernel<bf16, VB>), grid, dim3(BT), 0, st, a, tiles);
    else hipLaunchKernelGGL((linscan_bwd_kernel<float, VB>), grid, dim3(BT), 0, st, a, tiles);
    return hipGetLastError();
}

hipError_t launch_linscan_step(const LinScanArgs& a, hipStream_t st) {
    constexpr int V = 4;
    const int64_t work = (int64_t)a.N * ((a.C + V - 1) / V);
    const dim3 grid((unsigned)((work + BT - 1) / BT));
    if (a.dtype == 1) hipLaunchKernelGGL((linscan_step_kernel<bf16, V>), grid, dim3(BT), 0, st, a);
    else hipLaunchKernelGGL((linscan_step_kernel<float, V>), grid, dim3(BT), 0, st, a);
    return hipGetLastError();
}

}  // namespace kda
