// zi_orth_gemm.hip -- the products of the orthogonalised update (zi_orth.hip), on
// the MFMA kernel of zi_gemm.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zi_gemm.h"
#include "zi_internal.h"

namespace zi {
namespace {

int64_t min64(int64_t x, int64_t y) { return x < y ? x : y; }

// One product.  The tiles of a last, partial round of workgroups are each taken
// by several of them, as many as the round has room for, with at least kLeast
// steps of the reduction each: joining the pieces' sums costs as much as a few
// steps, more with larger tiles.  (1024 x 4096 on tiles of 64: 288 us with at
// least 8 steps, 338 with 32; 3008 x 3008 on tiles of 128: 912 with 16, 991
// with 8.)
template <bool Q_RS, int EPI, int B>
hipError_t run_product(OrthArgs a, hipStream_t s) {
    constexpr int TILE = 32 * B, kLeast = B == 2 ? 8 : 16, kMost = 16;
    constexpr int kGroup = B * B < 16 ? 16 / (B * B) : 1;  // pieces whose sums are read together
    const int tiles_p = (int)((a.rows + TILE - 1) / TILE), tiles_q = (int)((a.cols + TILE - 1) / TILE);
    const int64_t nt = EPI == EPI_APPLY ? (int64_t)tiles_p * tiles_q : (int64_t)tiles_p * (tiles_p + 1) / 2;
    const int64_t cap = kOrthUnits * (B == 8 ? 1 : B == 4 ? 2 : 4);
    const int64_t r = nt % cap;
    int64_t pieces = r ? min64(min64(cap / r, a.red / (BK * kLeast)), kMost) : 1;
    pieces = pieces / kGroup * kGroup;
    if (pieces < 2) pieces = 1;
    a.pieces = (int32_t)pieces;
    a.split_tail = pieces > 1 ? (int32_t)r : 0;
    const int64_t grid = nt + a.split_tail * (pieces - 1);
    if (a.red % BK != 0 || grid > INT32_MAX / kThreads) return hipErrorInvalidValue;
    hipLaunchKernelGGL((gemm_kernel<_Float16, Q_RS, false, EPI, true, B, B, false, OrthArgs>), dim3((unsigned)grid),
                       dim3(kThreads), 0, s, a, tiles_p, tiles_q);
    return hipGetLastError();
}
template <bool Q_RS, int EPI>
hipError_t run_sized(const OrthArgs &a, int tile, hipStream_t s) {
    return tile == 256   ? run_product<Q_RS, EPI, 8>(a, s)
           : tile == 128 ? run_product<Q_RS, EPI, 4>(a, s)
                         : run_product<Q_RS, EPI, 2>(a, s);
}

}  // namespace

hipError_t launch_orth(OrthOp op, int tile, const OrthArgs &a, hipStream_t stream) {
    switch (op) {
        case OrthOp::Gram:
            return run_sized<false, EPI_GRAM>(a, tile, stream);
        case OrthOp::Poly:
            return run_sized<false, EPI_POLY>(a, tile, stream);
        case OrthOp::Apply:
            return run_sized<true, EPI_APPLY>(a, tile, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace zi
