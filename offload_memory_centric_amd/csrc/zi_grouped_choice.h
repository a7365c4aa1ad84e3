// zi_grouped_choice.h -- which kernel a product grouped by expert runs on, by its sizes
// alone (zi_grouped.hip).  Host code without HIP, so that it is tested without a GPU.
#pragma once

#include <math.h>
#include <stdint.h>

namespace zi {
namespace {

inline int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
inline int64_t min64(int64_t x, int64_t y) { return x < y ? x : y; }

// A launch's threads, which are a signed 32-bit number here, in workgroups.
inline int64_t most_workgroups(int64_t threads) { return INT32_MAX / threads; }

// Workgroups of a product over the groups' rows (forward, dX), one a tile of tile_p rows
// by tile_q columns.  The groups' sizes are known on the device only: of row tiles there
// are at most total / tile_p and one more for every group with rows, and workgroups
// without a tile end at once.  (Eight at a time, one an XCD.)
inline int64_t row_grid(int64_t total, int64_t groups, int64_t cols, int64_t tile_p, int64_t tile_q) {
    return ceil_div((total / tile_p + min64(groups, total)) * ceil_div(cols, tile_q), 8) * 8;
}
// The same of the weight gradients, rows by cols each.
inline int64_t dw_grid(int64_t rows, int64_t cols, int64_t groups, int64_t tile) {
    return ceil_div(ceil_div(rows, tile) * ceil_div(cols, tile) * groups, 8) * 8;
}

// The macro-tile that takes least, and how long (us), by its rounds of workgroups on 256
// compute units, of which each holds one tile of 256, two of 128 or four of 64.  A round
// takes what the products of many shapes measured (us for a reduction of r thousand):
// 19.1 r + 14, 12.6 r + 0.3 r^2 + 6 and 12 r + 0.3 r^2 + 5; a tile that has its unit to
// itself 16.5 r + 14, 7.4 r + 5 and 6.2 r + 4.  (The smaller tiles of a long reduction
// drift apart and share less in the L2s: 13570 rows of 31 groups, 24320 x 2048, 1463 us
// with tiles of 256, 1773 with 128.)  A group's row tiles are estimated for sizes that
// fall off exponentially: one at least, and half of one unused where there are many.
// (8000 rows of 60 groups, 4096 x 1024: 196 us with 256, 158 with 128, as chosen; 20000
// of 16, 1024 x 1024: 74.0 and 60.8, and 83.7 with 64.  Over 45 products of 1 to 64 groups
// the choice takes 2 % longer than the best tile on average; equal sizes were not among them:
// 64 groups of 128 rows, which are 64 tiles of 128, count as 101.  The times themselves may be
// off by more: 14211 rows of 24 groups, 5000 x 2048, 319 us estimated and 371 to 388 measured.)
// Tiles of which a launch cannot have as many are not taken: grid(tile) workgroups.
struct TileChoice {
    int tile;  // 0: none
    double us;
};
template <typename Grid>
TileChoice tile_of(int64_t rows, int64_t cols, int64_t groups, double red, bool ragged, Grid &&grid) {
    const double r = red / 1000;
    TileChoice best = {0, 0};
    for (int tile = 256; tile >= 64; tile /= 2) {
        if (grid(tile) > most_workgroups(256)) break;
        const double row_tiles =
            (double)groups * (ragged ? 1 / (1 - exp(-(double)tile * (double)groups / (double)rows)) : (double)ceil_div(rows, tile));
        const double each = row_tiles * (double)ceil_div(cols, tile) / 256;  // tiles a compute unit
        double t;
        if (tile == 256) {
            t = each > 1 ? ceil(each - 0.05) * (19.1 * r + 14) : 16.5 * r + 14;
        } else if (tile == 128) {
            t = each > 1 ? fmax(1, ceil(each / 2 - 0.05)) * (12.6 * r + 0.3 * r * r + 6) : 7.4 * r + 5;
        } else {
            const double alone = 6.2 * r + 4, full = 12 * r + 0.3 * r * r + 5;
            t = each > 4 ? each / 4 * full : alone + (full - alone) * fmax(0, each - 1) / 3;
        }
        if (best.tile == 0 || t < 0.93 * best.us) best = {tile, t};  // where they are close, the larger
    }
    return best;
}

// Whether few_rows_kernel takes less than the best macro-tile: it reads W once for every
// 16 rows, at 8.7 TB/s from the L2s, and from memory at 5.1 TB/s, the macro-tiles at 4.2;
// a round of its workgroups takes 3 us besides.
// (us, few rows and best tile: 128 rows of 64 groups, 2048 x 1408, 72.1 and 98.7; 2 rows
// of 8, 8192 x 4096, 26.5, 56.3; 128 rows of 8, 4096 x 2048, 25.5, 36.0; 256 rows of them
// 45.2, 36.8.)
inline bool few_rows(int64_t R, int64_t K, int64_t M, int64_t live, double best_us) {
    if (row_grid(R, live, M, 16, 32) > most_workgroups(256)) return false;
    const double tiles = R <= 16 * live ? (double)live : (double)R / 16 + 0.5 * (double)live;
    const double weights = (double)live * (double)K * (double)M * 2e-6;  // MB
    const double groups = tiles * (double)ceil_div(M, 32);  // workgroups, of which a compute unit holds two
    const double t = fmax(3 * ceil(groups / 512), 5 + groups * 48 * (double)K * 2e-6 / 8.7);
    return fmax(t, weights / 5.1) < fmax(best_us, weights / 4.2);
}

// Whether few_rows_dx_kernel takes less than the best macro-tile: a workgroup takes 3 us
// and 1.2 ns for one of W's rows, all of them together their 64 bytes at 3.5 TB/s.  (us, few rows and
// best tile: 10 rows of one group, 9568 -> 6768, 28.2 and 63.5; 25 of 18, 6128 -> 88, 11.0
// and 25.5; one, 8192 -> 8192, 42.7 and 47.8; 32 rows of 64, 2048 -> 1408, 45.8 and 29.8;
// 500 of 4, 8192 -> 512, 53.0 and 57.5, of which it takes the tile.)
inline bool few_rows_dx(int64_t R, int64_t K, int64_t M, int64_t live, double best_us) {
    if (row_grid(R, live, K, 16, 32) > most_workgroups(512)) return false;
    const double row_tiles = R <= 16 * live ? (double)live : (double)R / 16 + 0.5 * (double)live;
    const double tiles = row_tiles * (double)ceil_div(K, 32);
    return 2 + fmax(ceil(tiles / 256) * (3 + 1.2e-3 * (double)M), 3 + tiles * 64e-6 / 3.5 * (double)M) < best_us;
}

// The macro-tile of a product, kFewRows for the kernels of few rows, 0 where a launch
// cannot have as many workgroups as any of them needs.
constexpr int kFewRows = 16;
inline int grouped_fwd_tile(int64_t R, int64_t K, int64_t M, int64_t E) {
    const int64_t live = min64(E, R);
    const TileChoice best = tile_of(R, M, live, (double)K, true, [&](int tile) { return row_grid(R, live, M, tile, tile); });
    return best.tile && few_rows(R, K, M, live, best.us) ? kFewRows : best.tile;
}
inline int grouped_dx_tile(int64_t R, int64_t K, int64_t M, int64_t E) {
    const int64_t live = min64(E, R);
    const TileChoice best = tile_of(R, K, live, (double)M, true, [&](int tile) { return row_grid(R, live, K, tile, tile); });
    return best.tile && few_rows_dx(R, K, M, live, best.us) ? kFewRows : best.tile;
}
// (An accumulating one has tiles of 256 alone.)
inline int grouped_dw_tile(int64_t R, int64_t K, int64_t M, int64_t E, bool accumulate) {
    auto grid = [&](int tile) { return dw_grid(M, K, E, tile); };
    if (accumulate) return grid(256) <= most_workgroups(256) ? 256 : 0;
    return tile_of(M, K, E, (double)R / (double)E, false, grid).tile;
}

}  // namespace
}  // namespace zi
