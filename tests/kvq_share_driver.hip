// Prints, for one sequence of a chunk call, what every row tile is allotted in the line of work (in
// 1/16 tiles), the tiles that it has and the allotments in front of it: host code of kvq_chunk.h.
//   kvq_share_driver ROWS TILE len kv group window
#include <stdio.h>
#include <stdlib.h>

#include "kvq_chunk.h"

using namespace onebit;

template <int ROWS, int TILE>
static void print(const KvqAttnArgs &a, const KvqSeq &s) {
    const ChunkShare share = chunk_share<ROWS, TILE>(a, s);
    for (int rt = 0; rt < share.row_tiles; ++rt) {
        int base;
        const int tiles = chunk_tiles<ROWS, TILE>(a, s, rt, base);
        printf("%lld %d %lld\n", (long long)share.of(rt), tiles, (long long)share.before(rt));
    }
    printf("end %d %lld\n", kSetupTiles, (long long)share.before(share.row_tiles));
}

int main(int argc, char **argv) {
    if (argc != 7) return 2;
    KvqAttnArgs a{};
    KvqSeq s{0, atoi(argv[3]), atoi(argv[4])};
    a.group = atoi(argv[5]);
    a.window = atoi(argv[6]);
    a.max_rows = 48;
    if (atoi(argv[2]) == 128)
        print<256, 128>(a, s);
    else if (atoi(argv[2]) == 64)
        print<256, 64>(a, s);
    else
        print<128, 32>(a, s);
    return 0;
}
