// zi_grouped_dx.hip -- the grouped input gradients (zi_grouped.hip) on the MFMA kernel.
#include "zi_grouped_gemm.h"

namespace zi {
namespace {

template <typename T>
hipError_t dispatch(int tile, const GroupArgs &a, hipStream_t s) {
    if (a.pre) return run_tiled<T, true, EPI_DACT>(a, tile, s);
    return a.out_f32 ? run_tiled<T, true, EPI_F32>(a, tile, s) : run_tiled<T, true, EPI_LP>(a, tile, s);
}

}  // namespace

hipError_t launch_grouped_dx(int dtype, int tile, const GroupArgs &a, hipStream_t s) {
    return dtype == 1 ? dispatch<_Float16>(tile, a, s) : dispatch<__bf16>(tile, a, s);
}

}  // namespace zi
