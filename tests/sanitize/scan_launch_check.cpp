// The scan's launches at the largest sizes the host accepts: fewer than 2^32
// threads each, with the workgroups for empty sequences.  Host arithmetic only.
#include <stdio.h>

#include "kda_block.hpp"

int main() {
    int bad = 0;
    for (int C = 1; C <= 1 << 20; C = C < 300 ? C + 1 : C + C / 7) {
        int64_t lo = 1, hi = (int64_t)1 << 32;  // accepted, refused
        while (hi - lo > 1) {
            const int64_t m = (lo + hi) / 2;
            (kda::linscan_fits(m, C) ? lo : hi) = m;
        }
        const kda::LinScanShape s = kda::linscan_shape((int32_t)(lo < 0x7fff0000 ? lo : 0x7fff0000), C);
        const int64_t threads = ((int64_t)s.tiles * s.cblocks + kda::LINSCAN_EMPTY) * s.waves * 64;
        if (threads >= (int64_t)1 << 32 || threads < (int64_t)1 << 20) {
            printf("C = %d: T = %lld takes %lld threads\n", C, (long long)lo, (long long)threads);
            ++bad;
        }
        if ((int64_t)s.tiles * s.waves * 16 < lo && lo <= 0x7fff0000) ++bad;   // the tiles hold every token,
        if ((int64_t)s.cblocks * 64 * s.vec < C) ++bad;                        // the blocks every column
        if (((size_t)s.tiles * C + (size_t)s.cblocks * kda::LINSCAN_LINE) * 8 > kda::linscan_chain_bytes(lo, C)) ++bad;  // the workspace every word
    }
    if (!bad) printf("scan launch check ok\n");
    return bad != 0;
}
