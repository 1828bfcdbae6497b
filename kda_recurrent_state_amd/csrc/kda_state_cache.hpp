// kda_state_cache.hpp -- host-side launcher of the 8-bit state cache.
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

}  // namespace kda
