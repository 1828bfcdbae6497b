// kda_rows.hpp -- building blocks of the row-wise kernels (norms, short
// convolution, diagonal recurrence): vector accesses without an alignment
// requirement, positions of packed tokens in their sequences, and the sum of
// partial rows.
#pragma once

#include "kda_device.hpp"

namespace kda {

// V consecutive elements of type T at any element-aligned address.  Global
// memory accesses on gfx950 need no more than the element's alignment, so a
// row that starts at an odd address takes the same instructions as an aligned
// one.
//
// Loading and converting are apart: a conversion waits for its load, so code
// that has several loads to make makes them all first.  For the same reason a
// lane whose V columns would pass the row's end does not branch to a shorter
// load: it takes the row's last V columns instead (column below), of which the
// first few belong to its neighbour too.  Both compute the same values from the
// same inputs and store the same bits.
template <typename T, int V> struct Pack {
    static constexpr int N = V * sizeof(T) <= 16 ? V : 16 / sizeof(T);  // elements of one access
    static_assert((N & (N - 1)) == 0 && V % N == 0, "an access is a power of two (a vector of 3 takes the room of 4)");
    typedef T vec __attribute__((vector_size(N * sizeof(T)), aligned(sizeof(T))));
    vec part[V / N];
    __device__ __forceinline__ float operator[](int i) const { return (float)part[i / N][i % N]; }
};

template <int V, typename T> __device__ __forceinline__ Pack<T, V> load_v(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <int V, typename T> __device__ __forceinline__ void store_v(T* p, const float (&v)[V]) {
    Pack<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.part[i / Pack<T, V>::N][i % Pack<T, V>::N] = from_f32<T>(v[i]);
    *reinterpret_cast<Pack<T, V>*>(p) = r;
}
template <int V> __device__ __forceinline__ void zero_v(float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = 0.f;
}
template <int V, typename T> __device__ __forceinline__ void get_v(const Pack<T, V>& r, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = r[i];
}
// The same past the caches: for data that is touched once.
template <int V, typename T> __device__ __forceinline__ Pack<T, V> load_nt(const T* p) {
    Pack<T, V> r;
#pragma unroll
    for (int k = 0; k < V / Pack<T, V>::N; ++k)
        r.part[k] = __builtin_nontemporal_load(reinterpret_cast<const typename Pack<T, V>::vec*>(p) + k);
    return r;
}
template <int V, typename T> __device__ __forceinline__ void store_nt(T* p, const float (&v)[V]) {
    typename Pack<T, V>::vec* q = reinterpret_cast<typename Pack<T, V>::vec*>(p);
#pragma unroll
    for (int k = 0; k < V / Pack<T, V>::N; ++k) {
        typename Pack<T, V>::vec r;
#pragma unroll
        for (int i = 0; i < Pack<T, V>::N; ++i) r[i] = from_f32<T>(v[k * Pack<T, V>::N + i]);
        __builtin_nontemporal_store(r, q + k);
    }
}

// Inputs that fill half of the 256 MiB last-level cache or more are read past it, and
// the call's outputs written past it: they would only push each other out.  Smaller
// ones may be there from whoever wrote them.  Measured, us through the cache and past
// it (three sets of inputs and outputs in turn), by the MiB of inputs:
//   convolution, bf16: 64: 25 and 30, 96: 41 and 41, 128: 55 and 53, 192: 78 and 74, 512:
//     193 and 185; its gradient, 96: 43 and 45, 128: 57 and 56, 512: 178 and 169
//   gated norm: fp32, 37: 10.7 and 12.2; bf16, 64: 19.5 and 19.2, 128: 38 and 34, 512: 135
//     and 126; its gradient, 192: 68 and 65, 768: 249 and 240
//   residual norm, gradient, bf16, 384: 133 and 118
// The convolution and the scan write past it at every size.  With the call that reads the
// output behind them in a graph, ordinary stores took, us against these: convolution, then
// scan, by the MiB of the output, 16: 29.5 and 28.6, 64: 89 and 92; convolution, then
// norm, 8: 13.5 and 12.8, 64: 54 and 57; scan, then norm, 8: 21.1 and 20.2, 32: 53.7 and 52.1,
// 64: 87.2 and 88.0.
inline bool past_cache(int64_t in_bytes) { return in_bytes >= 128ll << 20; }
// (An access of two halves touches each line twice, which has to stay cached in between.)
template <bool PAST, int V, typename T> __device__ __forceinline__ Pack<T, V> load_c(const T* p) {
    if constexpr (PAST && V * sizeof(T) <= 16) return load_nt<V>(p);
    else return load_v<V>(p);
}
template <bool PAST, int V, typename T> __device__ __forceinline__ void store_c(T* p, const float (&v)[V]) {
    if constexpr (PAST && V * sizeof(T) <= 16) store_nt<V>(p, v);
    else store_v<V>(p, v);
}

// First column of the lane whose columns start at c, in a row of C >= V.
template <int V> __host__ __device__ __forceinline__ int column(int c, int C) { return c + V <= C ? c : C - V; }

// The channel of thread j of a block of 64 V columns, and whether it is the thread's own:
// a lane that was moved back from the row's end, or that lies past it, carries channels
// of other lanes' too.
struct ChainColumn { int c; bool owner; };
template <int V> __host__ __device__ __forceinline__ ChainColumn chain_column(int cb, int j, int C) {
    const int at = (cb * 64 + j / V) * V, c = column<V>(at, C) + j % V;
    return {c, c >= at};
}

// Sequences of a packed axis of T tokens: offsets cu[0..N] on the device, or
// (cu null) N sequences of eq tokens each.  Offsets are clamped to [0, T], so
// that no offset, whatever it holds, reaches outside the tensors.
struct Seqs {
    const int32_t* cu;
    int32_t N;
    int32_t T;
    int32_t eq;
    __device__ __forceinline__ int start(int n) const {
        if (!cu) return n * eq;
        if (n == 0) return 0;
        const int s = cu[n];
        return s < 0 ? 0 : (s > T ? T : s);
    }
    __device__ __forceinline__ int end() const { return start(N); }
    // The sequence of token t (0 <= t < end()): the last n with start(n) <= t.
    __device__ __forceinline__ int find(int t) const {
        if (!cu) return t / eq;
        int lo = 0, hi = N;  // start(lo) <= t, answer in [lo, hi)
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (start(m) <= t) lo = m; else hi = m;
        }
        return lo;
    }
};

// The sequence of a token by a whole wavefront (all lanes active, t the same in
// each): the lanes read 64 offsets at once, where Seqs::find reads them one
// after the other.  Offsets out of order give some sequence in [0, N).
__device__ __forceinline__ int wave_find(const Seqs& sq, int t) {
    if (!sq.cu) return t / sq.eq;
    const int lane = threadIdx.x % WAVE;
    int lo = 0, hi = sq.N;
    while (hi - lo > 1) {
        const int step = (hi - lo + WAVE - 1) / WAVE, n = lo + (lane + 1) * step;
        const int below = __popcll(__ballot(n < hi && sq.start(n < hi ? n : lo) <= t));
        lo += below * step;
        hi = hi - lo < step ? hi : lo + step;
    }
    return lo;
}

// By the exponential and reciprocal instructions: within (|z| + 6) 2^-24 of itself.
__device__ __forceinline__ float sigmoid_f(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// Sum over the G (a power of two up to 64) consecutive lanes of a group.
template <int G>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int m = 1; m < G; m <<= 1) x += __shfl_xor(x, m);
    return x;
}

}  // namespace kda
