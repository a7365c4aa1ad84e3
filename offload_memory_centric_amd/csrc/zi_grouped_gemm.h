// zi_grouped_gemm.h -- launches of the grouped products on the MFMA kernel of
// zi_gemm.h, one product to a source file.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zi_gemm.h"
#include "zi_grouped_choice.h"
#include "zi_internal.h"

namespace zi {
namespace {

// One workgroup a macro-tile (row_grid and dw_grid, which the choice of the tile keeps
// within a launch's bounds).
template <typename T, bool Q_RS, bool P_RS, int EPI, bool ALIGNED, int B>
hipError_t run_grouped(const GroupArgs &a, hipStream_t s) {
    constexpr int TILE = 32 * B;
    constexpr bool DW = Q_RS && P_RS;
    const int64_t tiles_q = ceil_div(a.cols, TILE);
    const int64_t tiles_p = DW ? ceil_div(a.rows, TILE) : a.total / TILE + min64(a.groups, a.total);
    const int64_t grid = DW ? dw_grid(a.rows, a.cols, a.groups, TILE) : row_grid(a.total, a.groups, a.cols, TILE, TILE);
    if (grid <= 0) return hipSuccess;
    if (grid > most_workgroups(kThreads)) return hipErrorInvalidValue;
    // a lane's offset inside a tile or a step stays below the descriptors' range
    if (a.ldq > kGroupLd || a.ldp > kGroupLd || a.red >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
    hipLaunchKernelGGL((gemm_kernel<T, Q_RS, P_RS, EPI, ALIGNED, B, B, false, GroupArgs>), dim3((unsigned)grid), dim3(kThreads), 0, s,
                       a, (int)tiles_p, (int)tiles_q);
    return hipGetLastError();
}

// Tiles of 64 are for products that wait for memory and launches, not for the matrix
// cores: they have the one form that checks the reduction's end.
template <typename T, bool Q_RS, int EPI>
hipError_t run_tiled(const GroupArgs &a, int tile, hipStream_t s) {
    const bool aligned = a.red % BK == 0;
    if (tile == 64) return run_grouped<T, Q_RS, false, EPI, false, 2>(a, s);
    if (tile == 128)
        return aligned ? run_grouped<T, Q_RS, false, EPI, true, 4>(a, s) : run_grouped<T, Q_RS, false, EPI, false, 4>(a, s);
    return aligned ? run_grouped<T, Q_RS, false, EPI, true, 8>(a, s) : run_grouped<T, Q_RS, false, EPI, false, 8>(a, s);
}

}  // namespace
}  // namespace zi
