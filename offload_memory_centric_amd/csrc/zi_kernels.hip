// zi_kernels.hip -- gfx950 kernels of the tiled linear operator: the products of
// a weight tile (zi_gemm.h) and the elementwise GeLU backward.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "zi_gemm.h"
#include "zi_internal.h"

namespace zi {
namespace {

// ---- GeLU -------------------------------------------------------------------------

// GeLU(a) = a * Phi(a), Phi(a) = erfc(-a / sqrt 2) / 2 (exact erf form), in
// fp64.  The forward epilogue rounds it once to 16 bits, and its input is a
// 16-bit value, so it is a table of 65536 entries per type, built once per
// device (build_gelu_table) and looked up from LDS in the epilogue.
__device__ __forceinline__ double gelu_f64(double a) { return a * (0.5 * erfc(-a / sqrt(2.0))); }

// double -> float rounded to odd (truncate, then set the last bit if
// inexact): a later round-to-nearest-even to a format at least two bits
// narrower then gives the correctly rounded result of the double.
__device__ __forceinline__ float round_to_odd_f32(double h) {
    float f = (float)h;
    if ((double)f != h) {
        uint32_t u = __builtin_bit_cast(uint32_t, f);
        if (fabs((double)f) > fabs(h)) u -= 1;  // rounded away from zero: one step back
        f = __builtin_bit_cast(float, u | 1u);
    }
    return f;
}

__device__ uint16_t g_gelu_f16[65536];
__device__ uint16_t g_gelu_bf16[65536];

template <>
__device__ __forceinline__ uint16_t *gelu_table<_Float16>() { return g_gelu_f16; }
template <>
__device__ __forceinline__ uint16_t *gelu_table<__bf16>() { return g_gelu_bf16; }

template <typename T>
__global__ __launch_bounds__(256) void gelu_table_kernel() {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    gelu_table<T>()[i] = (uint16_t)bits16<T>(round_to_odd_f32(gelu_f64((double)value16<T>(i))));
}

// GeLU'(a) = Phi(a) + a * phi(a), phi(a) = exp(-a^2 / 2) / sqrt(2 pi).
__device__ __forceinline__ float gelu_grad_f32(float a) {
    const float cdf = 0.5f * erfcf(-a * 0.70710678118654752f);
    const float pdf = 0.39894228040143268f * expf(-0.5f * a * a);
    return cdf + a * pdf;
}

// GeLU' in fp32 of every 16-bit input, built once per device with the
// function above (so a lookup gives the bits an evaluation would), for the
// GeLU backward.
__device__ float g_gelu_grad_f16[65536];
__device__ float g_gelu_grad_bf16[65536];

template <typename T>
__device__ __forceinline__ float *gelu_grad_table();
template <>
__device__ __forceinline__ float *gelu_grad_table<_Float16>() { return g_gelu_grad_f16; }
template <>
__device__ __forceinline__ float *gelu_grad_table<__bf16>() { return g_gelu_grad_bf16; }

template <typename T>
__global__ __launch_bounds__(256) void gelu_grad_table_kernel() {
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    gelu_grad_table<T>()[i] = gelu_grad_f32(value16<T>(i));
}

// ---- dA = RNE(dH * GeLU'(A)) ----------------------------------------------------------

// dA = RNE(dH * GeLU'(A)) with GeLU' looked up rather than evaluated: the
// evaluation (erfc and exp, tens of instructions per element) held the
// kernel at half the HBM rate.  A workgroup of 1024 threads (one per compute
// unit, with its LDS) copies the table's entries for |A| < 16 (both signs,
// kLim codes each: 152 KiB for fp16, 131 KiB for bf16) into LDS and reads the
// rest, which Gaussian-like data almost never holds, from the global table.
// OUT_F32: dA is written as the fp32 product itself, the value the 16-bit
// form rounds once.
template <typename T>
constexpr uint32_t gelu_grad_lim() { return std::is_same<T, _Float16>::value ? 0x4C00u : 0x4180u; }  // code of 16.0

template <typename T, bool OUT_F32>
__global__ __launch_bounds__(1024) void gelu_bwd_kernel(const float *__restrict__ dH,
                                                        const uint16_t *__restrict__ A,
                                                        void *__restrict__ dA, int64_t count) {
    constexpr uint32_t kLim = gelu_grad_lim<T>();
    static_assert(kLim % 4 == 0 && 2 * kLim * 4 <= 160 * 1024, "LDS table");
    __shared__ __attribute__((aligned(16))) float tab[2 * kLim];
    const float *gtab = gelu_grad_table<T>();
    for (uint32_t e = threadIdx.x * 4; e < 2 * kLim; e += blockDim.x * 4) {  // codes [0, kLim), [0x8000, +kLim)
        const uint32_t c = e < kLim ? e : 0x8000u + (e - kLim);
        *reinterpret_cast<f32x4 *>(tab + e) = *reinterpret_cast<const f32x4 *>(gtab + c);
    }
    __syncthreads();
    auto grad = [&](uint32_t c) __attribute__((always_inline)) -> float {
        const uint32_t m = c & 0x7fffu;
        return m < kLim ? tab[(c >> 15) * kLim + m] : gtab[c];
    };
    const int64_t stride = (int64_t)gridDim.x * blockDim.x * 8;
    uint16_t *dA16 = static_cast<uint16_t *>(dA);
    float *dA32 = static_cast<float *>(dA);
    for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 8; i < count; i += stride) {
        if (i + 8 <= count) {
            const f32x4 g0 = *reinterpret_cast<const f32x4 *>(dH + i);
            const f32x4 g1 = *reinterpret_cast<const f32x4 *>(dH + i + 4);
            const u32x4 av = *reinterpret_cast<const u32x4 *>(A + i);
            const float g[8] = {g0[0], g0[1], g0[2], g0[3], g1[0], g1[1], g1[2], g1[3]};
            float r[8];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                r[2 * w] = g[2 * w] * grad(av[w] & 0xffffu);
                r[2 * w + 1] = g[2 * w + 1] * grad(av[w] >> 16);
            }
            // the product is rounded to fp32 first and then, once, to 16 bits:
            // kept from fusing into a mixed-precision multiply that would
            // round the exact product straight to 16 bits
#pragma unroll
            for (int e = 0; e < 8; ++e) asm volatile("" : "+v"(r[e]));
            if constexpr (OUT_F32) {
                *reinterpret_cast<f32x4 *>(dA32 + i) = f32x4{r[0], r[1], r[2], r[3]};
                *reinterpret_cast<f32x4 *>(dA32 + i + 4) = f32x4{r[4], r[5], r[6], r[7]};
            } else {
                u32x4 o;
#pragma unroll
                for (int w = 0; w < 4; ++w) o[w] = bits16<T>(r[2 * w]) | (bits16<T>(r[2 * w + 1]) << 16);
                *reinterpret_cast<u32x4 *>(dA16 + i) = o;
            }
        } else {
            for (int64_t e = i; e < count; ++e) {
                float r = dH[e] * grad(A[e]);
                asm volatile("" : "+v"(r));
                if constexpr (OUT_F32)
                    dA32[e] = r;
                else
                    dA16[e] = (uint16_t)bits16<T>(r);
            }
        }
    }
}

// Launch shapes (per-wave blocks of q, p).  A product takes the 256 x 256
// tile unless a 320-wide tile covers its tile width (the forward's q extent,
// the gradient's p extent) with clearly less padding: the down-projection's
// 1600-column tiles fill 6.25 tiles of 256 but exactly 5 of 320.  (A 320 x 128
// forward tile, which at T = 32768 would fill five whole rounds of workgroups
// on 256 compute units where 320 x 192 leaves the fourth a third full, ran
// 14 % slower: 80 MFMAs per step do not cover the step's barrier and copies.)
enum Shape { SHAPE_8x8 = 0, SHAPE_10x6 = 1, SHAPE_6x10 = 2 };

int64_t padded(int64_t x, int64_t t) { return (x + t - 1) / t * t; }

Shape shape_for(GemmOp op, int64_t rows, int64_t cols) {
    const int64_t a88 = padded(cols, 256) * padded(rows, 256);
    if (op == GemmOp::Fwd) {
        const int64_t a = padded(cols, 320) * padded(rows, 192);
        if (a * 50 < a88 * 49) return SHAPE_10x6;
    } else if (op == GemmOp::Dw) {
        const int64_t a = padded(cols, 192) * padded(rows, 320);
        if (a * 50 < a88 * 49) return SHAPE_6x10;
    }
    return SHAPE_8x8;
}

template <typename T, bool Q_RS, bool P_RS, int EPI, int QB, int PB>
hipError_t run_shape(const GemmArgs &a, hipStream_t s) {
    const int tiles_p = (int)((a.rows + 32 * PB - 1) / (32 * PB));
    const int tiles_q = (int)((a.cols + 32 * QB - 1) / (32 * QB));
    const int64_t nt = (int64_t)tiles_p * tiles_q;
    if (nt <= 0) return hipSuccess;
    // the kernel counts reduction indices in 32 bits
    if (a.red < 1 || a.red >= ((int64_t)1 << 30)) return hipErrorInvalidValue;
    // a second weight tile: reduction rows from qsplit on (gradient products),
    // or output columns from qsplit on (forward products), which no
    // workgroup's columns may straddle
    if (a.Q2) {
        if (Q_RS && (a.qsplit <= 0 || a.qsplit % BK != 0 || a.qsplit >= a.red)) return hipErrorInvalidValue;
        if (!Q_RS && (a.qsplit <= 0 || a.qsplit % (32 * QB) != 0 || a.qsplit >= a.cols)) return hipErrorInvalidValue;
    }
    // the accumulating epilogue addresses 16 rows of C through one descriptor
    if (EPI == EPI_ACC && (a.ldc < 0 || (16 * a.ldc + 256) * 4 >= (int64_t)kNumRecords)) return hipErrorInvalidValue;
    // persistent workgroups: a grid of wg_cap (a multiple of 8, so that each
    // workgroup's tiles stay on its XCD) when there are more tiles than that
    if (a.wg_cap < 0 || a.wg_cap % 8 != 0) return hipErrorInvalidValue;
    if constexpr (EPI == EPI_ACC) {
        if (a.wg_cap > 0 && nt > a.wg_cap) {
            const dim3 g((unsigned)a.wg_cap);
            if (a.red % BK == 0)
                hipLaunchKernelGGL((gemm_kernel<T, Q_RS, P_RS, EPI, true, QB, PB, true>), g, dim3(kThreads), 0, s, a,
                                   tiles_p, tiles_q);
            else
                hipLaunchKernelGGL((gemm_kernel<T, Q_RS, P_RS, EPI, false, QB, PB, true>), g, dim3(kThreads), 0, s,
                                   a, tiles_p, tiles_q);
            return hipGetLastError();
        }
    }
    // GeLU forward: when the last round of tiles would leave at least half
    // of the compute units idle, its tiles run as two half-reductions each
    GemmArgs b = a;
    b.split_tail = 0;
    if constexpr (EPI == EPI_GELU || EPI == EPI_GELU_F32A) {
        if (a.split_part && a.split_cnt && a.split_cap > 0 && a.red % (2 * BK) == 0) {
            const int64_t r = nt % a.split_cap;
            if (r > 0 && 2 * r <= a.split_cap && r <= kSplitTiles) b.split_tail = (int32_t)r;
        }
    }
    const dim3 g((unsigned)(nt + b.split_tail));
    if (a.red % BK == 0)
        hipLaunchKernelGGL((gemm_kernel<T, Q_RS, P_RS, EPI, true, QB, PB, false>), g, dim3(kThreads), 0, s, b,
                           tiles_p, tiles_q);
    else
        hipLaunchKernelGGL((gemm_kernel<T, Q_RS, P_RS, EPI, false, QB, PB, false>), g, dim3(kThreads), 0, s, b,
                           tiles_p, tiles_q);
    return hipGetLastError();
}

template <typename T, bool Q_RS, bool P_RS, int EPI>
hipError_t run(GemmOp op, const GemmArgs &a, hipStream_t s) {
    // the forward (both operands reduction-contiguous) may take 320 x 192,
    // the gradient (both reduction-strided) 192 x 320
    if constexpr ((EPI == EPI_LP || EPI == EPI_F32) && !Q_RS && !P_RS) {
        if (shape_for(op, a.rows, a.cols) == SHAPE_10x6) return run_shape<T, Q_RS, P_RS, EPI, 10, 6>(a, s);
    }
    if constexpr ((EPI == EPI_LP || EPI == EPI_F32) && Q_RS && P_RS) {
        if (shape_for(op, a.rows, a.cols) == SHAPE_6x10) return run_shape<T, Q_RS, P_RS, EPI, 6, 10>(a, s);
    }
    return run_shape<T, Q_RS, P_RS, EPI, 8, 8>(a, s);
}

template <typename T>
hipError_t dispatch(GemmOp op, const GemmArgs &a, hipStream_t s) {
    switch (op) {
        case GemmOp::Fwd:
            return a.out_f32 ? run<T, false, false, EPI_F32>(op, a, s) : run<T, false, false, EPI_LP>(op, a, s);
        case GemmOp::FwdGelu:
            return a.out_f32 ? run<T, false, false, EPI_GELU_F32A>(op, a, s) : run<T, false, false, EPI_GELU>(op, a, s);
        case GemmOp::Dx:
            return run<T, true, false, EPI_ACC>(op, a, s);
        case GemmOp::Dw:
            return a.out_f32 ? run<T, true, true, EPI_F32>(op, a, s) : run<T, true, true, EPI_LP>(op, a, s);
    }
    return hipErrorInvalidValue;
}

}  // namespace

void gemm_tile(GemmOp op, int64_t rows, int64_t cols, int *tile_rows, int *tile_cols) {
    const Shape sh = (op == GemmOp::Fwd || op == GemmOp::Dw) ? shape_for(op, rows, cols) : SHAPE_8x8;
    *tile_cols = sh == SHAPE_10x6 ? 320 : (sh == SHAPE_6x10 ? 192 : 256);
    *tile_rows = sh == SHAPE_10x6 ? 192 : (sh == SHAPE_6x10 ? 320 : 256);
}

int64_t gemm_workgroups(GemmOp op, int64_t rows, int64_t cols) {
    int tp = 256, tq = 256;
    gemm_tile(op, rows, cols, &tp, &tq);
    return ((rows + tp - 1) / tp) * ((cols + tq - 1) / tq);
}

hipError_t launch_gemm(GemmOp op, int dtype, const GemmArgs &a, hipStream_t stream) {
    if (dtype == 1) return dispatch<_Float16>(op, a, stream);
    if (dtype == 2) return dispatch<__bf16>(op, a, stream);
    return hipErrorInvalidValue;
}

hipError_t build_gelu_tables(hipStream_t stream) {
    hipLaunchKernelGGL(gelu_table_kernel<_Float16>, dim3(256), dim3(256), 0, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(gelu_table_kernel<__bf16>, dim3(256), dim3(256), 0, stream);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(gelu_grad_table_kernel<_Float16>, dim3(256), dim3(256), 0, stream);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(gelu_grad_table_kernel<__bf16>, dim3(256), dim3(256), 0, stream);
    return hipGetLastError();
}

hipError_t launch_gelu_bwd(int dtype, const float *dH, const void *A, void *dA, int64_t count,
                           bool out_f32, hipStream_t stream) {
    if (count <= 0) return hipSuccess;
    // one workgroup of 1024 threads per compute unit (each holds the LDS
    // table), fewer for small counts
    const int64_t threads = (count + 7) / 8;
    int64_t blocks = (threads + 1023) / 1024;
    if (blocks > 256) blocks = 256;
    const uint16_t *a16 = static_cast<const uint16_t *>(A);
    const dim3 g((unsigned)blocks), b(1024);
    if (dtype == 1 && !out_f32)
        hipLaunchKernelGGL((gelu_bwd_kernel<_Float16, false>), g, b, 0, stream, dH, a16, dA, count);
    else if (dtype == 1)
        hipLaunchKernelGGL((gelu_bwd_kernel<_Float16, true>), g, b, 0, stream, dH, a16, dA, count);
    else if (dtype == 2 && !out_f32)
        hipLaunchKernelGGL((gelu_bwd_kernel<__bf16, false>), g, b, 0, stream, dH, a16, dA, count);
    else if (dtype == 2)
        hipLaunchKernelGGL((gelu_bwd_kernel<__bf16, true>), g, b, 0, stream, dH, a16, dA, count);
    else
        return hipErrorInvalidValue;
    return hipGetLastError();
}

}  // namespace zi
