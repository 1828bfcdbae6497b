// kda_state_cache.hip -- recurrent states in 8 bits: quantised as they are written to a cache's slots, and read back.
//
// A row of W values has one scale, s = max |x| (1 / M) in fp32 (M = 127 for int8, 448 for e4m3; 1 / M the
// nearest fp32 value), and codes that are the nearest of the format's values to the exact quotient x / s,
// ties to even: the division's own rounding never decides.
//
// Both directions move 5 bytes a value.  A row lies in 1 to 64 neighbouring lanes, 4 values each (16 bytes in, 4 out), and
// a thread has 4 rows on their way.  256 states of 32 x 128 x 128 (672 MB each way): reading 118 us, 5.7 TB/s, bound by
// memory; writing 169 us, 4.0 TB/s, 88 of them vector issue (26 instructions a value, most of them the test for borders).
// The same states over and over, so that some are still in the last-level cache: int8 148 us written, e4m3 151, and 185
// where rows' values span five orders of magnitude and most quads hold one below 2^-6 of the scale's unit, which is divided.
#include "kda_state_cache.hpp"

#include "kda_rows.hpp"

namespace kda {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ uint32_t pack_i8(const float (&q)[4]) {  // whole numbers or NaN (a scale that is no number: 0 x scale is NaN)
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= ((uint32_t)(int)__builtin_amdgcn_fmed3f(q[i], -127.f, 127.f) & 0xffu) << (8 * i);
    return w;
}
__device__ __forceinline__ uint32_t pack_f8(const float (&v)[4]) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = v[i] != v[i] ? v[i] : __builtin_amdgcn_fmed3f(v[i], -448.f, 448.f);
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
}
// Four codes.  x (1 / s) by the reciprocal instruction is within 3 units in the last place of x / s (the instruction's
// one may be two of the product's, which adds a half): it decides wherever it is further than 4 from a border, and the division is only made
// where one of a wavefront's is not, or the reciprocal of s is not finite.  43 vector instructions a value with
// every division made were 192 us for 134e6 values, where memory takes 130.
__device__ __forceinline__ uint32_t codes4(const float (&x)[4], float s, float inverse, bool f8) {
    float q[4];
    bool sure = s >= 0x1p-120f;  // false for NaN
    if (f8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[i] = x[i] * inverse;
            // of 20 bits behind a code's own three the border has the first; below 2^-6 borders lie elsewhere
            const uint32_t b = __float_as_uint(q[i]) & 0x7fffffffu;
            const uint32_t from = (b & 0xfffffu) - 0x7fffcu;
            sure = sure && from > 8u && (b >= 0x3c800004u || b == 0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = x[i] * inverse, near = rintf(v);
            sure = sure && fabsf(v - near) < 0.49995f;  // 4 units of 2^-17, those of 64 to 128, are 3.1e-5
            q[i] = near;
        }
    }
    if (!sure) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float v = beside_border(x[i], s);
            q[i] = f8 ? v : v != v ? 0.f : rintf(v);
        }
    }
    return f8 ? pack_f8(q) : pack_i8(q);
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

// The largest over 2^log2 neighbouring lanes, in each: exchanges within 16 lanes need no trip through LDS.
template <int CTRL> __device__ __forceinline__ uint32_t lane_of(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 15, 15, false);
}
__device__ __forceinline__ uint32_t lanes_max(uint32_t v, int log2) {
    if (log2 > 0) v = max(v, lane_of<0xb1>(v));   // quad_perm 1, 0, 3, 2
    if (log2 > 1) v = max(v, lane_of<0x4e>(v));   // quad_perm 2, 3, 0, 1
    if (log2 > 2) v = max(v, lane_of<0x141>(v));  // mirrored in 8 lanes: the other four
    if (log2 > 3) v = max(v, lane_of<0x140>(v));  // mirrored in 16: the other eight
    if (log2 > 4) v = max(v, (uint32_t)__shfl_xor((int)v, 16));
    if (log2 > 5) v = max(v, (uint32_t)__shfl_xor((int)v, 32));
    return v;
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
    const int lanes = 1 << lanes_log2, cl = threadIdx.x & (lanes - 1), rows_at_once = NT >> lanes_log2;
    const bool f8 = a.format == 1;
    const float unit = f8 ? 1.f / 448.f : 1.f / 127.f;
    const float* src = a.values_in + (int64_t)r * a.rows * a.width;
    int64_t row0 = (int64_t)blk * rows_at_once * U + (threadIdx.x >> lanes_log2);
    Row<NV> x[U];
    auto load = [&]() {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * rows_at_once;
            if (row < a.rows) x[u].load(src + row * a.width, a.width, cl, lanes);
        }
    };
    load();  // on its way while the slots are looked through
    const int slot = slot_of(a, r);
    if (slot < 0) return;
    if (a.slots) {
        int again = 0;
        for (int j = r + 1 + threadIdx.x; j < a.states; j += NT) again |= a.slots[j] == slot;
        if (__syncthreads_or(again)) return;
    }
    uint8_t* dst = a.codes + (int64_t)slot * a.rows * a.width;
    float* scales = a.scales + (int64_t)slot * a.rows;
    while (row0 < a.rows) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = row0 + u * rows_at_once;
            // the largest magnitude as whole numbers, so that a NaN is larger than everything
            uint32_t most = 0;
#pragma unroll
            for (int k = 0; k < NV; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) most = max(most, __float_as_uint(x[u].v[k][i]) & 0x7fffffffu);
            most = lanes_max(most, lanes_log2);
            if (row >= a.rows) continue;
            const float scale = __uint_as_float(most) * unit, inverse = __builtin_amdgcn_rcpf(scale);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int c = (k * lanes + cl) * 4;
                if (c >= a.width) continue;
                const uint32_t w = scale == 0.f ? 0u : codes4(x[u].v[k], scale, inverse, f8);
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
        row0 += (int64_t)blocks * rows_at_once * U;
        load();
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
    // rows in flight a thread, write + read of 256 states of 4096 rows of 128, us: 2 198 + 121, 4 169 + 118, 8 299 + 130
    if (nv <= 1) return launch<1, 4>(a, write, log2, st);
    if (nv <= 4) return launch<4, 1>(a, write, log2, st);
    return launch<32, 1>(a, write, log2, st);
}

}  // namespace kda
