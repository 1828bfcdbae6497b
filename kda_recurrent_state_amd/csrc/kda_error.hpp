// kda_error.hpp -- status reporting shared by the files that define C entry points.
#pragma once

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/kda.h"

namespace kda {

// Text of the last error of this thread (kda_last_error).
inline thread_local char g_last_error[256] = "";

inline int fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline int fail(int status, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return status;
}

inline int ok() {
    g_last_error[0] = '\0';
    return KDA_OK;
}

// Non-null pointers with the alignment the kernels' accesses need.
inline int check_ptrs(const void* const* ptrs, const char* const* names, const int* align, int count) {
    for (int i = 0; i < count; ++i) {
        if (!ptrs[i]) return fail(KDA_ERR_INVALID_ARGUMENT, "%s is NULL", names[i]);
        if ((uintptr_t)ptrs[i] % (uintptr_t)align[i])
            return fail(KDA_ERR_MISALIGNED, "%s is not %d-byte aligned", names[i], align[i]);
    }
    return KDA_OK;
}

}  // namespace kda
