// Whether a tensor whose tokens lie apart has a byte in a range: against every byte, for all small shapes.
// Host arithmetic only.
#include <stdio.h>

#include "kda_checks.hpp"

int main() {
    using namespace kda::checks;
    long checked = 0;
    const int64_t base = 100;
    for (int64_t tokens = 0; tokens <= 4; ++tokens)
        for (int64_t bytes = 1; bytes <= 6; ++bytes)
            for (int64_t step = bytes; step <= bytes + 7; ++step)
                for (int64_t a = base - 8; a < base + 60; ++a)
                    for (int64_t b = a; b < a + 14; ++b) {
                        bool want = false;
                        for (int64_t t = 0; t < tokens; ++t)
                            for (int64_t i = 0; i < bytes; ++i) {
                                const int64_t at = base + t * step + i;
                                want = want || (at >= a && at < b);
                            }
                        const Extent e{"t", reinterpret_cast<const void*>(base), tokens, step, bytes};
                        const bool got = a < b && touches(e, (uintptr_t)a, (uintptr_t)b);
                        ++checked;
                        if (got != want) {
                            printf("%ld tokens of %ld, %ld apart: [%ld, %ld) gives %d\n", (long)tokens, (long)bytes, (long)step,
                                   (long)(a - base), (long)(b - base), got);
                            return 1;
                        }
                    }
    const Extent none = whole("none", nullptr, 8);
    if (touches(none, 0, 1000)) return 1;
    // far apart: no product passes 64 bits
    const Extent far{"far", reinterpret_cast<const void*>(base), 0x7fff0000, int64_t(1) << 42, 8};
    if (touches(far, uintptr_t(1) << 60, (uintptr_t(1) << 60) + 8) || !touches(far, uintptr_t(1) << 45, uintptr_t(1) << 46)) return 1;
    printf("extent check ok: %ld ranges\n", checked);
    return 0;
}
