// zi_stream.h -- products of a few rows, whose operands go from memory straight to the
// matrix cores' registers: what such a product waits for is the bytes of its larger
// operand, which LDS would only delay.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "zi_gemm.h"

namespace zi {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// v_mfma_f32_16x16x32 for code whose waits the compiler sees to.
template <typename T>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mfma<_Float16>(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mfma<__bf16>(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (int)kNumRecords, (int)kRsrcWord3);
}

// The offsets of a lane's part (16 bytes of row lane % 16, the (lane / 16)-th of a
// step's four) of F fragments of 16 rows each, `rows` of which there are.
template <int F>
__device__ __forceinline__ void fragment_offsets(int64_t rows, int64_t ld, uint32_t (&off)[F]) {
    const int r = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int f = 0; f < F; ++f) off[f] = 16 * f + r < rows ? (uint32_t)(((16 * f + r) * ld + 8 * g) * 2) : kOOB;
}

// acc += Q P^T over the steps [s0, s1) of 32 reduction values, `red` in all: QF
// fragments of 16 rows of Q, PF of P, AHEAD steps' loads in flight while as many are
// multiplied.  Lane l gets column l % 16 of P and rows 4 (l / 16) .. +3 of Q.
template <typename T, int QF, int PF, int AHEAD>
__device__ __forceinline__ void stream_product(__amdgpu_buffer_rsrc_t qr, const uint32_t (&qo)[QF], __amdgpu_buffer_rsrc_t pr,
                                               const uint32_t (&po)[PF], int s0, int s1, int red, f32x4 (&acc)[QF][PF]) {
    const int g = (threadIdx.x & 63) >> 4;
    u32x4 q[2][AHEAD][QF], p[2][AHEAD][PF];
    auto load = [&](auto B_, int s) __attribute__((always_inline)) {
        constexpr int b = decltype(B_)::value;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            // past the last step or the reduction's end: zeros (two offsets past the
            // descriptor's range stay past it when added)
            const uint32_t at = s + u < s1 && (s + u) * 32 + 8 * g < red ? (uint32_t)(s + u) * 64 : kOOB;
#pragma unroll
            for (int f = 0; f < QF; ++f)
                q[b][u][f] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(qr, (int)(qo[f] + at), 0, 0));
#pragma unroll
            for (int f = 0; f < PF; ++f)
                p[b][u][f] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(pr, (int)(po[f] + at), 0, 0));
        }
    };
    auto multiply = [&](auto B_) __attribute__((always_inline)) {
        constexpr int b = decltype(B_)::value;
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
            for (int i = 0; i < QF; ++i)
#pragma unroll
                for (int j = 0; j < PF; ++j) acc[i][j] = mfma<T>(q[b][u][i], p[b][u][j], acc[i][j]);
    };
    using B0 = std::integral_constant<int, 0>;
    using B1 = std::integral_constant<int, 1>;
    load(B0{}, s0);
    for (int s = s0; s < s1; s += 2 * AHEAD) {
        load(B1{}, s + AHEAD);
        multiply(B0{});
        if (s + 2 * AHEAD < s1) load(B0{}, s + 2 * AHEAD);
        multiply(B1{});
    }
    // The compiler has read the sums right behind the loop, before the last product
    // was in them (the build's assembly check looks for that).
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 7\n\ts_nop 7" ::: "memory");
}

}  // namespace
}  // namespace zi
