// The choice of the grouped products' kernels: for every line "op R K M E" of the
// standard input (op: fwd, dx, dw, acc) the tile, its workgroups and their threads.
#include "../../offload_memory_centric_amd/csrc/zi_grouped_choice.h"

#include <stdio.h>
#include <string.h>

int main() {
    char op[8];
    long long R, K, M, E;
    while (scanf("%7s %lld %lld %lld %lld", op, &R, &K, &M, &E) == 5) {
        using namespace zi;
        const bool fwd = !strcmp(op, "fwd"), dx = !strcmp(op, "dx");
        const int tile = fwd ? grouped_fwd_tile(R, K, M, E) : dx ? grouped_dx_tile(R, K, M, E) : grouped_dw_tile(R, K, M, E, op[0] == 'a');
        const long long cols = fwd ? M : K;
        const long long grid = !tile                ? 0
                               : !fwd && !dx        ? dw_grid(M, K, E, tile)
                               : tile == kFewRows ? row_grid(R, E, cols, 16, 32)
                                                    : row_grid(R, E, cols, tile, tile);
        printf("%d %lld %d\n", tile, grid, tile == kFewRows && dx ? 512 : 256);
    }
    return 0;
}
