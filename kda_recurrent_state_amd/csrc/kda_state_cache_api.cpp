// kda_state_cache_api.cpp -- the extern "C" entry points of the 8-bit state cache
// (include/kda.h): argument validation and launch.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/kda.h"
#include "kda_checks.hpp"
#include "kda_state_cache.hpp"

using namespace kda::checks;

namespace {

// A write looks through the slots of the states behind each of its own: 2^20 states look at 2^39 slots.
constexpr int kMaxStates = 1 << 20;

int check(const kda_state_cache_dims_t* d, const void* values, const char* name, const void* codes, const float* scales,
          const int32_t* slots, kda::StateCacheArgs* a) {
    if (!d) return fail(KDA_ERR_INVALID_ARGUMENT, "dims is NULL");
    if (d->states < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "states = %d < 0", d->states);
    if (d->states > kMaxStates) return fail(KDA_ERR_INVALID_ARGUMENT, "states = %d: at most %d", d->states, kMaxStates);
    if (d->slots < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "slots = %d < 0", d->slots);
    if (d->rows < 0 || d->rows > (int64_t)1 << 40)
        return fail(KDA_ERR_INVALID_ARGUMENT, "rows = %lld: must be 0 to 2^40", (long long)d->rows);
    if (d->width < 1) return fail(KDA_ERR_INVALID_ARGUMENT, "width = %d < 1", d->width);
    if (d->width > kda::STATE_CACHE_MAX_WIDTH)
        return fail(KDA_ERR_UNSUPPORTED, "width = %d: at most %d", d->width, kda::STATE_CACHE_MAX_WIDTH);
    if ((double)d->rows * d->width * (d->states > d->slots ? d->states : d->slots) > 0x1p60)
        return fail(KDA_ERR_INVALID_ARGUMENT, "states, slots, rows and width = %d, %d, %lld and %d are too large", d->states,
                    d->slots, (long long)d->rows, d->width);
    if (d->format != KDA_CACHE_I8 && d->format != KDA_CACHE_E4M3)
        return fail(KDA_ERR_INVALID_ARGUMENT, "format = %d is not KDA_CACHE_I8 or KDA_CACHE_E4M3", d->format);
    if (d->reserved != 0) return fail(KDA_ERR_INVALID_ARGUMENT, "reserved = %d is not 0", d->reserved);
    *a = kda::StateCacheArgs();
    a->states = d->states;
    a->num_slots = d->slots;
    a->rows = d->rows;
    a->width = d->width;
    a->format = d->format == KDA_CACHE_E4M3;
    if (!slots && d->states > d->slots)
        return fail(KDA_ERR_INVALID_ARGUMENT, "slots is NULL but %d states do not fit %d slots", d->states, d->slots);
    KDA_TRY(check_optional(slots, 4, "slots"));
    const void* ptrs[] = {values, codes, scales};
    const char* names[] = {name, "codes", "scales"};
    const int align[] = {4, 1, 4};
    const bool any = d->states > 0 && d->rows > 0;
    KDA_TRY(check_ptrs(ptrs, names, align, !any ? 0 : d->slots > 0 ? 3 : 1));
    a->codes = const_cast<uint8_t*>(static_cast<const uint8_t*>(codes));
    a->scales = const_cast<float*>(scales);
    a->slots = slots;
    return KDA_OK;
}

}  // namespace

extern "C" {

int kda_state_cache_write(const kda_state_cache_dims_t* d, const float* states, const int32_t* slots, void* codes,
                          float* scales, void* stream) {
    kda::StateCacheArgs a;
    KDA_TRY(check(d, states, "states", codes, scales, slots, &a));
    a.values_in = states;
    return hip_status(kda::launch_state_cache(a, true, (hipStream_t)stream), "state cache write");
}

int kda_state_cache_read(const kda_state_cache_dims_t* d, const void* codes, const float* scales, const int32_t* slots,
                         float* states, void* stream) {
    kda::StateCacheArgs a;
    KDA_TRY(check(d, states, "states", codes, scales, slots, &a));
    a.values_out = states;
    return hip_status(kda::launch_state_cache(a, false, (hipStream_t)stream), "state cache read");
}

}  // extern "C"
