// zi_grouped_fwd.hip -- the grouped forward products (zi_grouped.hip) on the MFMA kernel.
#include "zi_grouped_gemm.h"

namespace zi {
namespace {

template <typename T>
hipError_t dispatch(int tile, const GroupArgs &a, hipStream_t s) {
    if (a.act) return run_tiled<T, false, EPI_ACT>(a, tile, s);
    return a.out_f32 ? run_tiled<T, false, EPI_F32>(a, tile, s) : run_tiled<T, false, EPI_LP>(a, tile, s);
}

}  // namespace

hipError_t launch_grouped_fwd(int dtype, int tile, const GroupArgs &a, hipStream_t s) {
    return dtype == 1 ? dispatch<_Float16>(tile, a, s) : dispatch<__bf16>(tile, a, s);
}

}  // namespace zi
