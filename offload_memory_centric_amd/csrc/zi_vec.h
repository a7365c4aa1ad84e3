// zi_vec.h -- device helpers of the row kernels (layer norm, embedding):
// vectors of eight elements of fp32, fp16 or bf16, held as fp32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/zi.h"

namespace zi {

typedef _Float16 f16_t;
typedef __bf16 bf16_t;

// Rows start wherever their stride puts them, so vectors are only as aligned
// as their elements; the hardware's global loads and stores take any address.
typedef uint16_t u16x8_u __attribute__((ext_vector_type(8), aligned(2)));
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));

template <typename T>
__device__ __forceinline__ float to_f32(uint16_t b) {
    return (float)__builtin_bit_cast(T, b);
}

// Eight consecutive elements.
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const f32x4_u a = *reinterpret_cast<const f32x4_u *>(p), b = *reinterpret_cast<const f32x4_u *>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = a[e];
        v[4 + e] = b[e];
    }
}
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    const u16x8_u a = *reinterpret_cast<const u16x8_u *>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32<T>(a[e]);
}

// One round to nearest even into T (none for fp32).
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
    *reinterpret_cast<f32x4_u *>(p) = f32x4_u{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4_u *>(p + 4) = f32x4_u{v[4], v[5], v[6], v[7]};
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    u16x8_u a;
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = __builtin_bit_cast(uint16_t, (T)v[e]);
    *reinterpret_cast<u16x8_u *>(p) = a;
}

// The first n (any n; nothing at or below 0) of eight elements; the others
// read as zero, and nothing past the n-th is touched.
template <typename T>
__device__ __forceinline__ void load_n(const T *p, int64_t n, float (&v)[8]) {
    if (n >= 8) {
        load8(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = e < n ? (float)p[e] : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store_n(T *p, int64_t n, const float (&v)[8]) {
    if (n >= 8) {
        store8(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) p[e] = (T)v[e];
    }
}

// The same store past the caches (nontemporal), for outputs that are written
// once.  Of fp32 values each of the two stores fills half of every line that
// the wave touches, and the caches are left to join them.
__device__ __forceinline__ void stream8(float *p, const float (&v)[8]) { store8(p, v); }
template <typename T>
__device__ __forceinline__ void stream8(T *p, const float (&v)[8]) {
    u16x8_u a;
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = __builtin_bit_cast(uint16_t, (T)v[e]);
    __builtin_nontemporal_store(a, reinterpret_cast<u16x8_u *>(p));
}

// Eight elements as they lie in memory: half the registers of their fp32
// values where the type is 16 bits wide.  16-bit elements are read past the
// caches, as they are written (stream8).
template <typename T>
struct Raw8 {
    u32x4_u v;
    __device__ __forceinline__ void load(const T *p) { v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_u *>(p)); }
    __device__ __forceinline__ float operator[](int e) const { return to_f32<T>((uint16_t)(v[e >> 1] >> (16 * (e & 1)))); }
    // Hides where the value comes from, so that what was computed from it
    // before is computed again rather than kept in registers.
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(v)); }
};
template <>
struct Raw8<float> {
    f32x4_u v[2];
    __device__ __forceinline__ void load(const float *p) {
        v[0] = *reinterpret_cast<const f32x4_u *>(p);
        v[1] = *reinterpret_cast<const f32x4_u *>(p + 4);
    }
    __device__ __forceinline__ float operator[](int e) const { return v[e >> 2][e & 3]; }
    __device__ __forceinline__ void forget() { asm volatile("" : "+v"(v[0]), "+v"(v[1])); }
};

// All of eight vectors are loaded at this point: none of their loads is put off
// until its value is needed.
template <typename T>
__device__ __forceinline__ void hold(Raw8<T> (&u)[8]) {
    asm volatile(""
                 : "+v"(u[0].v), "+v"(u[1].v), "+v"(u[2].v), "+v"(u[3].v), "+v"(u[4].v), "+v"(u[5].v), "+v"(u[6].v),
                   "+v"(u[7].v));
}
__device__ __forceinline__ void hold(Raw8<float> (&u)[8]) {
    asm volatile(""
                 : "+v"(u[0].v[0]), "+v"(u[0].v[1]), "+v"(u[1].v[0]), "+v"(u[1].v[1]), "+v"(u[2].v[0]), "+v"(u[2].v[1]),
                   "+v"(u[3].v[0]), "+v"(u[3].v[1]), "+v"(u[4].v[0]), "+v"(u[4].v[1]), "+v"(u[5].v[0]), "+v"(u[5].v[1]),
                   "+v"(u[6].v[0]), "+v"(u[6].v[1]), "+v"(u[7].v[0]), "+v"(u[7].v[1]));
}

// Eight elements of an array whose type is known at run time only (the same
// for every lane).
__device__ __forceinline__ void load8(const void *p, int dtype, int at, float (&v)[8]) {
    if (dtype == ZI_F32) {
        load8(static_cast<const float *>(p) + at, v);
        return;
    }
    const u32x4_u a = *reinterpret_cast<const u32x4_u *>(static_cast<const uint16_t *>(p) + at);
    if (dtype == ZI_F16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = to_f32<f16_t>((uint16_t)(a[e >> 1] >> (16 * (e & 1))));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = to_f32<bf16_t>((uint16_t)(a[e >> 1] >> (16 * (e & 1))));
    }
}

// load_n of an array whose type is known at run time only (the same for
// every lane).
__device__ __forceinline__ void load_n(const void *p, int dtype, int64_t at, int64_t n, float (&v)[8]) {
    if (dtype == ZI_F32)
        load_n(static_cast<const float *>(p) + at, n, v);
    else if (dtype == ZI_F16)
        load_n(static_cast<const f16_t *>(p) + at, n, v);
    else
        load_n(static_cast<const bf16_t *>(p) + at, n, v);
}

// Sum over groups of N consecutive lanes (N a power of two, at most 64); every
// lane gets it.
template <int N>
__device__ __forceinline__ float lane_sum(float x) {
#pragma unroll
    for (int m = 1; m < N; m <<= 1) x += __shfl_xor(x, m, 64);
    return x;
}

}  // namespace zi
