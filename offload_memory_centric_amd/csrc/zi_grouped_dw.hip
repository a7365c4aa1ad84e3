// zi_grouped_dw.hip -- the grouped weight gradients (zi_grouped.hip) on the MFMA
// kernel.  The reduction runs over a group's rows, so its end is always checked.
#include "zi_grouped_gemm.h"

namespace zi {
namespace {

template <typename T, int EPI>
hipError_t sized(int tile, const GroupArgs &a, hipStream_t s) {
    return tile == 256   ? run_grouped<T, true, true, EPI, false, 8>(a, s)
           : tile == 128 ? run_grouped<T, true, true, EPI, false, 4>(a, s)
                         : run_grouped<T, true, true, EPI, false, 2>(a, s);
}

template <typename T>
hipError_t dispatch(int tile, const GroupArgs &a, hipStream_t s) {
    if (a.accumulate) return run_grouped<T, true, true, EPI_ACC, false, 8>(a, s);
    return a.out_f32 ? sized<T, EPI_F32>(tile, a, s) : sized<T, EPI_LP>(tile, a, s);
}

}  // namespace

hipError_t launch_grouped_dw(int dtype, int tile, const GroupArgs &a, hipStream_t s) {
    return dtype == 1 ? dispatch<_Float16>(tile, a, s) : dispatch<__bf16>(tile, a, s);
}

}  // namespace zi
