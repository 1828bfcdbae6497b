// kda_state_cache.hip -- recurrent states in 8 bits: quantised as they are written to a cache's slots, and read back.
//
// A row of W values has one scale, s = max |x| (1 / M) in fp32 (M = 127 for int8, 448 for e4m3; 1 / M the
// nearest fp32 value), and codes that are the nearest of the format's values to the exact quotient x / s,
// ties to even: the division's own rounding never decides.  Both directions move 5 bytes a value and a few operations; memory bounds them.
#include "kda_state_cache.hpp"

#include "kda_rows.hpp"

namespace kda {
namespace {

constexpr int NT = 256;

// The code of the quotient x / s, s > 0.  The division is correctly rounded to fp32; where it lands on a
// border between two codes without being one, the sign of the remainder says which side x / s is on.
// (Every border has at most 12 significant bits, so a quotient with more is none.)
__device__ __forceinline__ float beside_border(float x, float s) {
    const float q = x / s;
    const uint32_t b = __float_as_uint(q);
    if ((b & 0xfffu) == 0) {
        const float rest = fmaf(-q, s, x);
        if (rest != 0.f) return __uint_as_float((rest > 0.f) == (q > 0.f) ? b + 1 : b - 1);
    }
    return q;
}
__device__ __forceinline__ uint32_t code_i8(float x, float s) {
    const float q = rintf(beside_border(x, s));
    return q != q ? 0u : (uint32_t)(int)fminf(fmaxf(q, -127.f), 127.f) & 0xffu;  // with a scale that is no number: 0 x scale is NaN
}
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float s, bool f8) {
    if (f8) {
        float q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = beside_border(x[i], s);
            q[i] = v != v ? v : fminf(fmaxf(v, -448.f), 448.f);
        }
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
    }
    return code_i8(x[0], s) | code_i8(x[1], s) << 8 | code_i8(x[2], s) << 16 | code_i8(x[3], s) << 24;
}
__device__ __forceinline__ void values4(uint32_t c, float s, bool f8, float (&v)[4]) {
    if (f8) {
        v[0] = __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
        v[1] = __builtin_amdgcn_cvt_f32_fp8((int)c, 1);
        v[2] = __builtin_amdgcn_cvt_f32_fp8((int)c, 2);
        v[3] = __builtin_amdgcn_cvt_f32_fp8((int)c, 3);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(c >> (8 * i));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= s;
}

__device__ __forceinline__ int slot_of(const StateCacheArgs& a, int r) {
    const int64_t s = a.slots ? a.slots[r] : r;
    return s >= 0 && s < a.num_slots ? (int)s : -1;
}

// The lanes of a row, NV accesses of 4 values each; a lane whose access would pass the row's end takes the
// row's last four values, a row of fewer than four is read one by one.
template <int NV> struct Row {
    float v[NV][4];
    __device__ __forceinline__ void load(const float* p, int W, int cl, int lanes) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * lanes + cl) * 4;
            zero_v(v[k]);
            if (W >= 4) {
                if (c < W) get_v(load_nt<4>(p + column<4>(c, W)), v[k]);
            } else if (c < W) {
                for (int i = 0; i < W; ++i) v[k][i] = p[i];
            }
        }
    }
};

// Workgroups (row block, state): the block's rows of the state go to the state's slot, unless a later
// state of the call has the same one.
template <int NV, int U>
__global__ void __launch_bounds__(NT) state_write_kernel(StateCacheArgs a, int lanes_log2, int blocks) {
    const int r = (int)(blockIdx.x / blocks), blk = (int)(blockIdx.x % blocks);
    const int slot = slot_of(a, r);
    if (slot < 0) return;
    if (a.slots) {
        int again = 0;
        for (int j = r + 1 + threadIdx.x; j < a.states; j += NT) again |= a.slots[j] == slot;
        if (__syncthreads_or(again)) return;
    }
    const int lanes = 1 << lanes_log2, cl = threadIdx.x & (lanes - 1), rows_at_once = NT >> lanes_log2;
    const bool f8 = a.format == 1;
    const float unit = f8 ? 1.f / 448.f : 1.f / 127.f;
    const float* src = a.values_in + (int64_t)r * a.rows * a.width;
    uint8_t* dst = a.codes + (int64_t)slot * a.rows * a.width;
    float* scales = a.scales + (int64_t)slot * a.rows;
    for (int64_t row0 = (int64_t)blk * rows_at_once * U + (threadIdx.x >> lanes_log2); row0 < a.rows;
         row0 += (int64_t)blocks * rows_at_once * U) {
        Row<NV> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * rows_at_once;
            if (row < a.rows) x[u].load(src + row * a.width, a.width, cl, lanes);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * rows_at_once;
            // the largest magnitude as whole numbers, so that a NaN is larger than everything
            uint32_t most = 0;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) most = max(most, __float_as_uint(x[u].v[k][i]) & 0x7fffffffu);
            for (int m = 1; m < lanes; m <<= 1) most = max(most, (uint32_t)__shfl_xor((int)most, m));
            if (row >= a.rows) continue;
            const float scale = __uint_as_float(most) * unit;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * lanes + cl) * 4;
                if (c >= a.width) continue;
                const uint32_t w = scale == 0.f ? 0u : codes4(x[u].v[k], scale, f8);
                uint8_t* p = dst + row * a.width;
                if (a.width >= 4) {
                    typedef uint32_t word __attribute__((aligned(1)));
                    __builtin_nontemporal_store(w, reinterpret_cast<word*>(p + column<4>(c, a.width)));
                } else {
                    for (int i = 0; i < a.width; ++i) p[i] = (uint8_t)(w >> (8 * i));
                }
            }
            if (cl == 0) scales[row] = scale;
        }
    }
}

template <int NV, int U>
__global__ void __launch_bounds__(NT) state_read_kernel(StateCacheArgs a, int lanes_log2, int blocks) {
    const int r = (int)(blockIdx.x / blocks), blk = (int)(blockIdx.x % blocks);
    const int slot = slot_of(a, r);
    const int lanes = 1 << lanes_log2, cl = threadIdx.x & (lanes - 1), rows_at_once = NT >> lanes_log2;
    const bool f8 = a.format == 1;
    const uint8_t* src = a.codes + (int64_t)(slot < 0 ? 0 : slot) * a.rows * a.width;
    const float* scales = a.scales + (int64_t)(slot < 0 ? 0 : slot) * a.rows;
    float* dst = a.values_out + (int64_t)r * a.rows * a.width;
    for (int64_t row0 = (int64_t)blk * rows_at_once * U + (threadIdx.x >> lanes_log2); row0 < a.rows;
         row0 += (int64_t)blocks * rows_at_once * U) {
        uint32_t w[U][NV];
        float s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * rows_at_once;
            s[u] = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) w[u][k] = 0;
            if (row >= a.rows || slot < 0) continue;
            s[u] = scales[row];
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * lanes + cl) * 4;
                if (c >= a.width) continue;
                const uint8_t* p = src + row * a.width;
                if (a.width >= 4) {
                    typedef uint32_t word __attribute__((aligned(1)));
                    w[u][k] = __builtin_nontemporal_load(reinterpret_cast<const word*>(p + column<4>(c, a.width)));
                } else {
                    for (int i = 0; i < a.width; ++i) w[u][k] |= (uint32_t)p[i] << (8 * i);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * rows_at_once;
            if (row >= a.rows) continue;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * lanes + cl) * 4;
                if (c >= a.width) continue;
                float v[4];
                values4(w[u][k], s[u], f8, v);
                float* p = dst + row * a.width;
                if (a.width >= 4) store_nt<4>(p + column<4>(c, a.width), v);
                else for (int i = 0; i < a.width; ++i) p[i] = v[i];
            }
        }
    }
}

template <int NV, int U> hipError_t launch(const StateCacheArgs& a, bool write, int log2, hipStream_t st) {
    const int at_once = (NT >> log2) * U;
    int64_t blocks = (a.rows + at_once - 1) / at_once;
    // a workgroup looks through the slots of the states behind its own once, so with many states it takes more rows
    const int64_t most = write && a.states > 4096 ? 1 : 0x7fffff / a.states > 0 ? 0x7fffff / a.states : 1;
    if (blocks > most) blocks = most;
    const dim3 grid((unsigned)(blocks * a.states));
    if (write) hipLaunchKernelGGL((state_write_kernel<NV, U>), grid, dim3(NT), 0, st, a, log2, (int)blocks);
    else hipLaunchKernelGGL((state_read_kernel<NV, U>), grid, dim3(NT), 0, st, a, log2, (int)blocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_state_cache(const StateCacheArgs& a, bool write, hipStream_t st) {
    if (a.states == 0 || a.rows == 0) return hipSuccess;
    const int quads = (a.width + 3) / 4;
    int log2 = 0;
    while ((1 << log2) < quads && log2 < 6) ++log2;
    const int nv = (quads + (1 << log2) - 1) >> log2;
    if (nv <= 1) return launch<1, 4>(a, write, log2, st);
    if (nv <= 4) return launch<4, 1>(a, write, log2, st);
    return launch<32, 1>(a, write, log2, st);
}

}  // namespace kda
