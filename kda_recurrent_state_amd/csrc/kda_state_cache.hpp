// kda_state_cache.hpp -- host-side launcher of the 8-bit state cache, and the quotient that its codes are taken from.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int STATE_CACHE_MAX_WIDTH = 8192;

struct StateCacheArgs {
    const float* values_in;  // write: [states][rows][width]
    float* values_out;       // read: the same
    uint8_t* codes;          // [num_slots][rows][width]
    float* scales;           // [num_slots][rows]
    const int32_t* slots;    // device, may be null (state r in slot r)
    int32_t states, num_slots;
    int64_t rows;            // rows of a state
    int32_t width, format;   // 0: int8, 1: e4m3
};
hipError_t launch_state_cache(const StateCacheArgs& a, bool write, hipStream_t st);

// The quotient x / s, s > 0, as a number on the same side of every border between two codes.  The division is correctly
// rounded to fp32; where it lands on a border without being one, the sign of the remainder says which side x / s is on.
// (Every border has at most 12 significant bits, so a quotient with more is none; nor is zero, to which a quotient
// below the least fp32 number is rounded.)  At a border a remainder is a multiple of the last place of s times that of the
// border, 2^-33 of the scale at the least, which a small scale would leave below fp32's range: both are moved up by a
// power of two (x is at most some hundred scales).
__host__ __device__ inline float beside_border(float x, float s) {
    const float up = s < 0x1p-60f ? 0x1p64f : 1.f;
    x *= up;
    s *= up;
    const float q = x / s, rest = __builtin_fmaf(-q, s, x);
    const uint32_t b = __builtin_bit_cast(uint32_t, q);
    const bool beside = (b & 0xfffu) == 0 && (b << 1) != 0 && rest != 0.f;
    return __builtin_bit_cast(float, b + (beside ? (rest > 0.f) == (q > 0.f) ? 1u : ~0u : 0u));
}

}  // namespace kda
