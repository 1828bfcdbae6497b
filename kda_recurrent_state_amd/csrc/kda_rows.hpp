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
template <typename T, int V> struct Pack;
template <> struct Pack<bf16, 8> { typedef __bf16 type __attribute__((vector_size(16), aligned(2))); };
template <> struct Pack<bf16, 4> { typedef __bf16 type __attribute__((vector_size(8), aligned(2))); };
template <> struct Pack<bf16, 2> { typedef __bf16 type __attribute__((vector_size(4), aligned(2))); };
template <> struct Pack<float, 4> { typedef float type __attribute__((vector_size(16), aligned(4))); };
template <> struct Pack<float, 2> { typedef float type __attribute__((vector_size(8), aligned(4))); };
template <> struct Pack<float, 8> {  // two 16-byte accesses
    struct type { Pack<float, 4>::type lo, hi; __device__ float operator[](int i) const { return i < 4 ? lo[i] : hi[i - 4]; } };
};

// The first n (any value; all if n >= V) of V elements at p; the rest are 0.
template <typename T, int V>
__device__ __forceinline__ void load_n(const T* p, int n, float (&v)[V]) {
    if (n >= V) {
        const typename Pack<T, V>::type r = *reinterpret_cast<const typename Pack<T, V>::type*>(p);
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = (float)r[i];
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < n ? (float)p[i] : 0.f;
    }
}

template <typename T, int V>
__device__ __forceinline__ void store_n(T* p, int n, const float (&v)[V]) {
    if (n >= V) {
        if constexpr (sizeof(T) * V > 16) {
            store_n<T, V / 2>(p, V / 2, reinterpret_cast<const float (&)[V / 2]>(v[0]));
            store_n<T, V / 2>(p + V / 2, V / 2, reinterpret_cast<const float (&)[V / 2]>(v[V / 2]));
        } else {
            typename Pack<T, V>::type r;
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = from_f32<T>(v[i]);
            *reinterpret_cast<typename Pack<T, V>::type*>(p) = r;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < n) p[i] = from_f32<T>(v[i]);
    }
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

__device__ __forceinline__ float sigmoid_f(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// Sum over the G (a power of two up to 64) consecutive lanes of a group.
template <int G>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int m = 1; m < G; m <<= 1) x += __shfl_xor(x, m);
    return x;
}

}  // namespace kda
