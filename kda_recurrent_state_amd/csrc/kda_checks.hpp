// kda_checks.hpp -- argument checks shared by the files that define the entry points of the
// operators around the state layer.
#pragma once

#include <hip/hip_runtime.h>

#include "kda_error.hpp"

namespace kda {
namespace checks {

using kda::check_ptrs;
using kda::fail;
using kda::ok;

constexpr int64_t kMaxTokens = 0x7fff0000;
constexpr int kMaxChannels = 1 << 20;
constexpr int kMaxWidth = 8192;
constexpr int64_t kMaxThreads = 0xffffffffll;  // threads of one launch along an axis

inline size_t round256(size_t x) { return (x + 255) / 256 * 256; }
inline int esize(int dtype) { return dtype == KDA_BF16 ? 2 : 4; }

inline int check_dtype(int dtype, const char* name) {
    if (dtype != KDA_F32 && dtype != KDA_BF16)
        return fail(KDA_ERR_INVALID_ARGUMENT, "%s = %d is not KDA_F32 or KDA_BF16", name, dtype);
    return KDA_OK;
}

// A token stride: 0 (contiguous) or at least the token's own elements.
inline int check_stride(int64_t* out, int64_t stride, int64_t least, const char* name) {
    if (stride == 0) stride = least;
    if (stride < least)
        return fail(KDA_ERR_INVALID_ARGUMENT, "%s = %lld is below the token's %lld elements", name, (long long)stride,
                    (long long)least);
    if (stride > (int64_t)1 << 40) return fail(KDA_ERR_INVALID_ARGUMENT, "%s = %lld is too large", name, (long long)stride);
    *out = stride;
    return KDA_OK;
}

// Sizes shared by the packed operators.
inline int check_packed(int32_t N, int64_t T, int32_t C, int32_t dtype, int32_t reserved) {
    if (N < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs = %d < 0", N);
    if (N > kMaxTokens) return fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs = %d: at most %lld", N, (long long)kMaxTokens);
    if (T < 0 || T > kMaxTokens)
        return fail(KDA_ERR_INVALID_ARGUMENT, "total_tokens = %lld: must be 0 to %lld", (long long)T,
                    (long long)kMaxTokens);
    if (C < 1 || C > kMaxChannels)
        return fail(KDA_ERR_INVALID_ARGUMENT, "channels = %d: must be 1 to %d", C, kMaxChannels);
    if (reserved != 0) return fail(KDA_ERR_INVALID_ARGUMENT, "reserved = %d is not 0", reserved);
    return check_dtype(dtype, "dtype");
}

inline int check_lengths(int32_t N, int64_t T, const int32_t* cu) {
    if (N == 0 && T != 0) return fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs = 0 but total_tokens = %lld", (long long)T);
    if (!cu && N > 0 && T % N != 0)
        return fail(KDA_ERR_INVALID_ARGUMENT,
                    "cu_seqlens is NULL but total_tokens = %lld is not a multiple of num_seqs = %d", (long long)T, N);
    if (cu && ((uintptr_t)cu & 3u)) return fail(KDA_ERR_MISALIGNED, "cu_seqlens is not 4-byte aligned");
    return KDA_OK;
}

inline int check_optional(const void* p, int align, const char* name) {
    if (p && (uintptr_t)p % (uintptr_t)align) return fail(KDA_ERR_MISALIGNED, "%s is not %d-byte aligned", name, align);
    return KDA_OK;
}

inline int check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return KDA_OK;
    if (!ws || have < need)
        return fail(KDA_ERR_INVALID_ARGUMENT, "needs a workspace of at least %zu bytes (got %zu)", need, ws ? have : (size_t)0);
    if ((uintptr_t)ws & 255u) return fail(KDA_ERR_MISALIGNED, "workspace is not 256-byte aligned");
    return KDA_OK;
}

// A tensor of a call: `tokens` of `bytes` bytes each, `step` bytes from one to the next.
struct Extent {
    const char* name;
    const void* p;  // may be null
    int64_t tokens, step, bytes;
};
inline Extent whole(const char* name, const void* p, int64_t bytes) { return {name, p, 1, bytes, bytes}; }

// Whether the tensor has a byte in [a, b); what lies between its tokens is not its own.
inline bool touches(const Extent& t, uintptr_t a, uintptr_t b) {
    const uintptr_t lo = (uintptr_t)t.p;
    if (!t.p || t.tokens <= 0 || lo >= b) return false;
    if (lo + (uintptr_t)t.bytes > a) return true;  // the first token
    const uintptr_t first = (a - lo - (uintptr_t)t.bytes) / (uintptr_t)t.step + 1;  // the first that ends behind a
    return first < (uintptr_t)t.tokens && lo + first * (uintptr_t)t.step < b;
}

// An output that lies on a tensor of the call that it may not (others[0 .. count)) is refused.
inline int check_apart(const char* name, const void* out, int64_t bytes, const Extent* others, int count) {
    const uintptr_t a = (uintptr_t)out, b = a + (uintptr_t)bytes;
    for (int i = 0; i < count; ++i)
        if (others[i].p != nullptr && touches(others[i], a, b))
            return fail(KDA_ERR_INVALID_ARGUMENT, "%s overlaps %s", name, others[i].name);
    return KDA_OK;
}

inline int hip_status(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
    return ok();
}

#define KDA_TRY(call)            \
    do {                         \
        const int st_ = (call);  \
        if (st_) return st_;     \
    } while (0)

}  // namespace checks
}  // namespace kda
