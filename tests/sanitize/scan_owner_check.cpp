// Who publishes a channel's word in the scan's chain: of all threads of a tile's
// column blocks that carry the channel (lanes at a row's end repeat its last
// columns), exactly one.  Host arithmetic only.
#include <stdio.h>

#include <vector>

#include "kda_block.hpp"
#include "kda_rows.hpp"

template <int V> static int check(int C) {
    const int cblocks = (C + 64 * V - 1) / (64 * V);
    std::vector<int> owners(C, 0), carriers(C, 0);
    for (int cb = 0; cb < cblocks; ++cb)
        for (int j = 0; j < 64 * V; ++j) {
            const kda::ChainColumn k = kda::chain_column<V>(cb, j, C);
            if (k.c < 0 || k.c >= C) return 1;
            ++carriers[k.c];
            owners[k.c] += k.owner;
        }
    for (int c = 0; c < C; ++c)
        if (owners[c] != 1 || carriers[c] < 1) {
            printf("V = %d, C = %d: channel %d has %d publishers among %d threads\n", V, C, c, owners[c], carriers[c]);
            return 1;
        }
    return 0;
}

int main() {
    int bad = check<1>(1);
    for (int C = 2; C <= 5000; ++C) bad += check<2>(C);
    if (!bad) printf("scan owner check ok\n");
    return bad != 0;
}
