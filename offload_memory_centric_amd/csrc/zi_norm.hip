// zi_norm.hip -- layer norm in front of a block, forward and backward.
//
// Forward, row by row (D elements):
//   S = RNE(X + R)                (R, the block's output before it, is optional)
//   mean = sum S / D,  var = sum (S - mean)^2 / D,  rstd = 1 / sqrt(var + eps)
//   Y = (S - mean) rstd gamma + beta
// Backward, with h = (S - mean) rstd and g = dY gamma:
//   dX = rstd (g - mean(g) - h mean(g h)) + dS
//   dgamma = sum over rows of dY h,  dbeta = sum over rows of dY
// All sums are held in fp32; a row's variance is summed from the differences to
// its mean, so that a large mean costs no digits; S, Y and dX are rounded once.
//
// A row is held in registers by NT threads, V vectors of eight elements each,
// so that it is read once: the kernels are bound by HBM.  Rows longer than
// the largest of these (and those shorter than one vector) take a form that
// reads the row again for each sum.
//
// Rows pass the caches (nontemporal): the forward of 32768 x 25600 fp16 rows
// with their residual, 6.7 GB, takes 1.20 ms so (5.6 TB/s) and 1.69 ms through
// them; the backward, 8.4 GB with dY in fp32, 1.51 ms (5.6 TB/s).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/zi.h"
#include "zi_host.h"
#include "zi_vec.h"

namespace {

using namespace zi;

struct NormArgs {
    int64_t T, D;
    int64_t ldx, ldr, lds, ldy;
    float eps, width;  // width: D, which sums are divided by (a constant row's mean is exact)
    int32_t p_dtype;
    const void *X, *R;  // forward inputs
    void *S, *Y;        // forward outputs; the backward reads S, and Y is dY
    const void *gamma, *beta;
    float *mean, *rstd;
    const void *dS;  // backward
    void *dX;
    float *part;  // [gridDim.x][2][D]: each workgroup's sums of dY h and of dY
};

// Sum over the NT threads that hold a row; every one of them gets it.  `slots`:
// LDS words (NT / 64 of them).  One barrier is enough where two sums that take
// turns use different words: a wave that writes one sum's words has passed the
// other's barrier, which no wave reaches before it has read this one's last.
template <int NT>
__device__ __forceinline__ float row_sum(float x, float *slots) {
    if constexpr (NT <= 64) return lane_sum<NT>(x);
    x = lane_sum<64>(x);
    if ((threadIdx.x & 63) == 0) slots[threadIdx.x >> 6] = x;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) s += slots[w];
    return s;
}

// Rows of a workgroup at a time.  Where fewer are left, the threads without one
// stop: they must not read another's, which may be overwritten in place.
template <int NT>
constexpr int kRows = NT < 256 ? 256 / NT : 1;
template <int NT>
constexpr int kBlock = NT < 256 ? 256 : NT;

// The vectors of one thread's share of a row of D >= 8 elements: vector c
// covers elements [at, at + 8), and the row's last one is moved back to end
// with the row, as are those past its end, so that every load and store is a
// whole vector and none needs a branch.  Elements that a vector shares with the
// one before it then have the same value in both threads; sums leave them out
// (own).  The first FULL vectors lie in the row as they are, for every D that
// takes this shape.
template <int NT, int FULL>
struct Share {
    int t, D;
    __device__ __forceinline__ int at(int c) const {
        const int i = (c * NT + t) * 8;
        return NT > 64 && c < FULL ? i : min(i, D - 8);
    }
    __device__ __forceinline__ bool own(int c, int e) const {
        return (NT > 64 && c < FULL) || at(c) + e >= (c * NT + t) * 8;
    }
};

template <typename XT, typename YT, bool RES, int NT, int V, int FULL>
__global__ __launch_bounds__(kBlock<NT>) void norm_fwd_kernel(NormArgs a) {
    __shared__ float slots[2][NT <= 64 ? 1 : NT / 64];
    const int sub = kRows<NT> == 1 ? 0 : threadIdx.x / NT;
    const Share<NT, FULL> my{kRows<NT> == 1 ? (int)threadIdx.x : (int)threadIdx.x % NT, (int)a.D};
    for (int64_t first = (int64_t)blockIdx.x * kRows<NT>; first < a.T; first += (int64_t)gridDim.x * kRows<NT>) {
        if (kRows<NT> > 1 && first + sub >= a.T) break;  // (row_sum: these threads share no other row's sum)
        const int64_t row = first + sub;
        const XT *x = static_cast<const XT *>(a.X) + row * a.ldx;
        const YT *r = static_cast<const YT *>(a.R) + row * a.ldr;
        XT *sp = static_cast<XT *>(a.S) + row * a.lds;
        YT *y = static_cast<YT *>(a.Y) + row * a.ldy;
        Raw8<XT> xr[V];
        Raw8<YT> rr[V];
#pragma unroll
        for (int c = 0; c < V; ++c) {
            xr[c].load(x + my.at(c));
            if constexpr (RES) rr[c].load(r + my.at(c));
        }
        float s[V][8], sum = 0.f;
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[c][e] = xr[c][e];
                // the statistics are those of the stored sum, which the backward reads
                if constexpr (RES) s[c][e] = (float)(XT)(s[c][e] + rr[c][e]);
                sum += my.own(c, e) ? s[c][e] : 0.f;
            }
        const float mean = row_sum<NT>(sum, slots[0]) / a.width;
        if constexpr (RES) {  // the row has been read: S may replace X or R
            if (a.S) {
#pragma unroll
                for (int c = 0; c < V; ++c) stream8(sp + my.at(c), s[c]);
            }
        }
        float sq = 0.f;
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[c][e] -= mean;
                sq += my.own(c, e) ? s[c][e] * s[c][e] : 0.f;
            }
        const float rstd = 1.0f / sqrtf(row_sum<NT>(sq, slots[1]) / a.width + a.eps);
        if (my.t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
#pragma unroll
        for (int c = 0; c < V; ++c) {
            float g[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) s[c][e] *= rstd;
            if (a.gamma) {
                load8(a.gamma, a.p_dtype, my.at(c), g);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[c][e] *= g[e];
            }
            if (a.beta) {
                load8(a.beta, a.p_dtype, my.at(c), g);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[c][e] += g[e];
            }
            stream8(y + my.at(c), s[c]);
        }
    }
}

// Rows of any length: three passes over the row, which the caches serve.
template <typename XT, typename YT, bool RES>
__global__ __launch_bounds__(1024) void norm_fwd_long_kernel(NormArgs a) {
    constexpr int NT = 1024;
    __shared__ float slots[2][NT / 64];
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const XT *x = static_cast<const XT *>(a.X) + row * a.ldx;
        const YT *r = static_cast<const YT *>(a.R) + row * a.ldr;
        XT *sp = static_cast<XT *>(a.S) + row * a.lds;
        YT *y = static_cast<YT *>(a.Y) + row * a.ldy;
        // the row's sum as stored; from the first pass on it may have replaced X or R
        auto value = [&](int64_t i, bool first, float (&s)[8]) __attribute__((always_inline)) {
            if (RES && a.S && !first) {
                load_n(sp + i, a.D - i, s);
                return;
            }
            load_n(x + i, a.D - i, s);
            if constexpr (RES) {
                float u[8];
                load_n(r + i, a.D - i, u);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = (float)(XT)(s[e] + u[e]);
            }
        };
        float s[8], sum = 0.f, sq = 0.f;
        for (int64_t i = threadIdx.x * 8; i < a.D; i += NT * 8) {
            value(i, true, s);
            if (RES && a.S) store_n(sp + i, a.D - i, s);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += s[e];
        }
        const float mean = row_sum<NT>(sum, slots[0]) / a.width;
        for (int64_t i = threadIdx.x * 8; i < a.D; i += NT * 8) {
            value(i, false, s);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (i + e < a.D) sq += (s[e] - mean) * (s[e] - mean);
        }
        const float rstd = 1.0f / sqrtf(row_sum<NT>(sq, slots[1]) / a.width + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
        for (int64_t i = threadIdx.x * 8; i < a.D; i += NT * 8) {
            float g[8], b[8];
            value(i, false, s);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = (s[e] - mean) * rstd;
            if (a.gamma) {
                load_n(a.gamma, a.p_dtype, i, a.D - i, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] *= g[e];
            }
            if (a.beta) {
                load_n(a.beta, a.p_dtype, i, a.D - i, b);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] += b[e];
            }
            store_n(y + i, a.D - i, s);
        }
    }
}

__device__ __forceinline__ void pin(float (&v)[8]) {
    asm volatile(""
                 : "+v"(v[0]), "+v"(v[1]), "+v"(v[2]), "+v"(v[3]), "+v"(v[4]), "+v"(v[5]), "+v"(v[6]), "+v"(v[7]));
}

// A workgroup takes rows blockIdx.x, + gridDim.x, ... (kRows of them at a time)
// and holds its sums of dY h and dY in registers over all of them, and gamma in
// LDS.  Between the two uses of a row it is held as it was read.
template <typename XT, typename YT, int NT, int V, int FULL>
__global__ __launch_bounds__(kBlock<NT>) void norm_bwd_kernel(NormArgs a) {
    __shared__ float slots[2][NT <= 64 ? 1 : NT / 64];
    extern __shared__ __attribute__((aligned(16))) float gam[];  // gamma, D elements
    // registers of a thread's vectors: where dS too would not fit beside the
    // sums, S and dY (256 with 512 threads), it is read after the row's sums
    constexpr bool LATE = V * 2 * (8 + 2 * sizeof(XT) + sizeof(YT)) > 224;
    const int sub = kRows<NT> == 1 ? 0 : threadIdx.x / NT;
    const Share<NT, FULL> my{kRows<NT> == 1 ? (int)threadIdx.x : (int)threadIdx.x % NT, (int)a.D};
    for (int i = threadIdx.x * 8; i < a.D; i += kBlock<NT> * 8) {
        float g[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 1.f;
        if (a.gamma) load8(a.gamma, a.p_dtype, min(i, (int)a.D - 8), g);
        store8(gam + min(i, (int)a.D - 8), g);
    }
    __syncthreads();
    float ag[V][8], ab[V][8];
#pragma unroll
    for (int c = 0; c < V; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) ag[c][e] = ab[c][e] = 0.f;
    for (int64_t first = (int64_t)blockIdx.x * kRows<NT>; first < a.T; first += (int64_t)gridDim.x * kRows<NT>) {
        if (kRows<NT> > 1 && first + sub >= a.T) break;  // (row_sum: these threads share no other row's sum)
        const int64_t row = first + sub;
        const XT *x = static_cast<const XT *>(a.S) + row * a.lds;
        const YT *dy = static_cast<const YT *>(a.Y) + row * a.ldy;
        const XT *ds = static_cast<const XT *>(a.dS) + row * a.ldr;
        XT *dx = static_cast<XT *>(a.dX) + row * a.ldx;
        Raw8<XT> xr[V], ur[V];
        Raw8<YT> dr[V];
#pragma unroll
        for (int c = 0; c < V; ++c) {
            xr[c].load(x + my.at(c));
            dr[c].load(dy + my.at(c));
        }
        const float mean = a.mean[row], rstd = a.rstd[row];
        if (!LATE && a.dS) {  // on its way during the sums
#pragma unroll
            for (int c = 0; c < V; ++c) ur[c].load(ds + my.at(c));
        }
        float sg = 0.f, sgh = 0.f;
#pragma unroll
        for (int c = 0; c < V; ++c) {
            float g[8];
            load8(gam + my.at(c), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = (xr[c][e] - mean) * rstd, d = dr[c][e], w = d * g[e];
                ag[c][e] += d * h;
                ab[c][e] += d;
                sg += my.own(c, e) ? w : 0.f;
                sgh += my.own(c, e) ? w * h : 0.f;
            }
            // all of this vector's sums are formed here: left to itself, the
            // compiler puts some off past the row's sums and keeps what they
            // need in registers (in scratch, for long rows)
            pin(ag[c]);
            pin(ab[c]);
            asm volatile("" : "+v"(sg), "+v"(sgh));
            xr[c].forget();
            dr[c].forget();
        }
        const float mg = row_sum<NT>(sg, slots[0]) / a.width;
        const float mgh = row_sum<NT>(sgh, slots[1]) / a.width;
        // dX may be dS, and vectors overlap at the row's end: all of dS has
        // been read before anything is written
        if (a.dS) {
            if constexpr (LATE) {
#pragma unroll
                for (int c = 0; c < V; ++c) ur[c].load(ds + my.at(c));
            }
#pragma unroll
            for (int c = 0; c < V; ++c) ur[c].forget();
            if constexpr (LATE) __syncthreads();
        }
#pragma unroll
        for (int c = 0; c < V; ++c) {
            float o[8], g[8];
            load8(gam + my.at(c), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = (xr[c][e] - mean) * rstd;
                o[e] = (dr[c][e] * g[e] - mg - h * mgh) * rstd;
                if (a.dS) o[e] += ur[c][e];
            }
            stream8(dx + my.at(c), o);
        }
    }
    if (!a.part) return;
    float *pg = a.part + (int64_t)blockIdx.x * 2 * a.D, *pb = pg + a.D;
    if constexpr (NT >= 256) {
#pragma unroll
        for (int c = 0; c < V; ++c) {
            store8(pg + my.at(c), ag[c]);
            store8(pb + my.at(c), ab[c]);
        }
    } else {  // the workgroup's rows are summed here, in order
        __shared__ float fold[256 * 8];
#pragma unroll
        for (int c = 0; c < V; ++c)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 8; ++e) fold[threadIdx.x * 8 + e] = w ? ab[c][e] : ag[c][e];
                __syncthreads();
                for (int j = threadIdx.x; j < NT * 8; j += 256) {
                    float s = 0.f;
                    for (int k = 0; k < kRows<NT>; ++k) s += fold[k * NT * 8 + j];
                    const int i = Share<NT, FULL>{j >> 3, (int)a.D}.at(c) + (j & 7);
                    (w ? pb : pg)[i] = s;
                }
            }
    }
}

// dX of rows of any length; dgamma and dbeta are left to norm_cols_kernel.
template <typename XT, typename YT>
__global__ __launch_bounds__(1024) void norm_bwd_long_kernel(NormArgs a) {
    constexpr int NT = 1024;
    __shared__ float slots[2][NT / 64];
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const XT *x = static_cast<const XT *>(a.S) + row * a.lds;
        const YT *dy = static_cast<const YT *>(a.Y) + row * a.ldy;
        const XT *ds = static_cast<const XT *>(a.dS) + row * a.ldr;
        XT *dx = static_cast<XT *>(a.dX) + row * a.ldx;
        const float mean = a.mean[row], rstd = a.rstd[row];
        auto value = [&](int64_t i, float (&h)[8], float (&d)[8]) __attribute__((always_inline)) {
            float g[8];
            load_n(x + i, a.D - i, h);
            load_n(dy + i, a.D - i, d);
            if (a.gamma) load_n(a.gamma, a.p_dtype, i, a.D - i, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[e] = (h[e] - mean) * rstd;
                if (a.gamma) d[e] *= g[e];
            }
        };
        float h[8], d[8], sg = 0.f, sgh = 0.f;
        for (int64_t i = threadIdx.x * 8; i < a.D; i += NT * 8) {
            value(i, h, d);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sg += d[e];
                sgh += d[e] * h[e];
            }
        }
        const float mg = row_sum<NT>(sg, slots[0]) / a.width;
        const float mgh = row_sum<NT>(sgh, slots[1]) / a.width;
        for (int64_t i = threadIdx.x * 8; i < a.D; i += NT * 8) {
            float u[8];
            value(i, h, d);
            if (a.dS) load_n(ds + i, a.D - i, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                d[e] = (d[e] - mg - h[e] * mgh) * rstd;
                if (a.dS) d[e] += u[e];
            }
            store_n(dx + i, a.D - i, d);
        }
    }
}

// Sums of dY h and dY over every gridDim.y-th row, 8 columns a thread (long
// rows only; runs before the dX kernel, which may overwrite dY).
template <typename XT, typename YT>
__global__ __launch_bounds__(256) void norm_cols_kernel(NormArgs a) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= a.D) return;
    float ag[8] = {}, ab[8] = {};
    for (int64_t row = blockIdx.y; row < a.T; row += gridDim.y) {
        float h[8], d[8];
        load_n(static_cast<const XT *>(a.S) + row * a.lds + i, a.D - i, h);
        load_n(static_cast<const YT *>(a.Y) + row * a.ldy + i, a.D - i, d);
        const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            ag[e] += d[e] * ((h[e] - mean) * rstd);
            ab[e] += d[e];
        }
    }
    float *pg = a.part + (int64_t)blockIdx.y * 2 * a.D;
    store_n(pg + i, a.D - i, ag);
    store_n(pg + a.D + i, a.D - i, ab);
}

// dgamma and dbeta from the partial sums, in a fixed order: 64 columns and 16
// shares of the partial sums a workgroup at a time.
__global__ __launch_bounds__(1024) void norm_fold_kernel(const float *part, int64_t D, int32_t parts, float *dgamma,
                                                         float *dbeta) {
    __shared__ float sum[16][64];
    const int lane = threadIdx.x & 63, share = threadIdx.x >> 6;
    for (int64_t first = (int64_t)blockIdx.x * 64; first < 2 * D; first += (int64_t)gridDim.x * 64) {
        const int64_t col = first + lane;  // of [dgamma, dbeta]
        float s = 0.f;
        if (col < 2 * D) {
            constexpr int U = 8;  // loads in flight
            for (int p = share; p < parts; p += 16 * U) {
                float v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) v[u] = part[min(p + 16 * u, parts - 1) * 2 * D + col];
#pragma unroll
                for (int u = 0; u < U; ++u) s += p + 16 * u < parts ? v[u] : 0.f;
            }
        }
        sum[share][lane] = s;
        __syncthreads();
        if (share == 0 && col < 2 * D) {
#pragma unroll
            for (int k = 1; k < 16; ++k) s += sum[k][lane];
            if (col < D) {
                if (dgamma) dgamma[col] = s;
            } else {
                if (dbeta) dbeta[col - D] = s;
            }
        }
        __syncthreads();
    }
}

// ---- launches ---------------------------------------------------------------------

int64_t min64(int64_t x, int64_t y) { return x < y ? x : y; }

constexpr int64_t kMostGroups = 1 << 20;  // workgroups of a launch (a grid ends below 2^32 threads)
constexpr int64_t kLeastHeld = 8, kMostHeld = 32768;  // rows that are held in registers

// Workgroups of the backward, each with its own partial sums: as many as run at
// once where the sums take most of a compute unit's registers, and up to four
// times as many for shorter rows.
int64_t parts_of(int64_t D) { return D > 8192 ? 256 : D > 4096 ? 512 : 1024; }

// f(NT, V, FULL) for the threads and vectors that hold a row of D elements.
// Rows over 16384 take 1024 threads in the forward (2 % faster than 512 with
// twice the vectors), which leaves too few registers for the backward's sums
// (1024 threads there: half as fast); up to there it is the other way round
// (1024 threads: the backward 3 to 6 % faster, the forward up to 12 % slower).
// Even so the backward's sums, S and dY alone fill the 256 registers of its widest
// rows where S or dY is fp32, and some spill: with both in fp32 8192 x 25600 takes
// 831 us (113 registers; 3.4 GB, 4.0 TB/s) and 8192 x 32768 1430 (309; 3.0 TB/s).
template <bool FWD, typename F>
hipError_t with_shape(int64_t D, F &&f) {
#define ZI_SHAPE(NT, V, FULL)     \
    if (D <= (int64_t)NT * V * 8) \
    return f(std::integral_constant<int, NT>{}, std::integral_constant<int, V>{}, std::integral_constant<int, FULL>{})
    ZI_SHAPE(16, 1, 0);
    ZI_SHAPE(64, 1, 0);
    ZI_SHAPE(64, 2, 1);
    ZI_SHAPE(256, 1, 0);
    ZI_SHAPE(256, 2, 1);
    ZI_SHAPE(512, 2, 1);
    if constexpr (FWD) {
        ZI_SHAPE(512, 4, 2);
        ZI_SHAPE(1024, 3, 2);
        ZI_SHAPE(1024, 4, 3);
    } else {
        ZI_SHAPE(1024, 2, 1);
        ZI_SHAPE(512, 6, 4);
        ZI_SHAPE(512, 7, 6);
        ZI_SHAPE(512, 8, 7);
    }
#undef ZI_SHAPE
    return hipErrorInvalidValue;
}

template <typename XT, typename YT, bool RES>
hipError_t run_fwd(const NormArgs &a, hipStream_t s) {
    if (a.D < kLeastHeld || a.D > kMostHeld) {
        hipLaunchKernelGGL((norm_fwd_long_kernel<XT, YT, RES>), dim3((unsigned)min64(a.T, kMostGroups)), dim3(1024), 0, s, a);
        return hipGetLastError();
    }
    return with_shape<true>(a.D, [&](auto nt, auto v, auto full) {
        constexpr int NT = decltype(nt)::value, V = decltype(v)::value, FULL = decltype(full)::value;
        const unsigned grid = (unsigned)min64((a.T + kRows<NT> - 1) / kRows<NT>, kMostGroups);
        hipLaunchKernelGGL((norm_fwd_kernel<XT, YT, RES, NT, V, FULL>), dim3(grid), dim3(kBlock<NT>), 0, s, a);
        return hipGetLastError();
    });
}

template <typename XT, typename YT>
hipError_t run_bwd(const NormArgs &a, float *dgamma, float *dbeta, hipStream_t s) {
    int parts = 0;
    hipError_t e = hipSuccess;
    if (a.T > 0 && (a.D < kLeastHeld || a.D > kMostHeld)) {
        if (a.part) {
            parts = (int)min64(a.T, 64);  // (at most parts_of)
            const dim3 grid((unsigned)((a.D + 2047) / 2048), (unsigned)parts);
            hipLaunchKernelGGL((norm_cols_kernel<XT, YT>), grid, dim3(256), 0, s, a);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        hipLaunchKernelGGL((norm_bwd_long_kernel<XT, YT>), dim3((unsigned)min64(a.T, kMostGroups)), dim3(1024), 0, s, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    } else if (a.T > 0) {
        e = with_shape<false>(a.D, [&](auto nt, auto v, auto full) {
            constexpr int NT = decltype(nt)::value, V = decltype(v)::value, FULL = decltype(full)::value;
            parts = (int)min64((a.T + kRows<NT> - 1) / kRows<NT>, parts_of(a.D));
            hipLaunchKernelGGL((norm_bwd_kernel<XT, YT, NT, V, FULL>), dim3((unsigned)parts), dim3(kBlock<NT>),
                               (unsigned)a.D * 4, s, a);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
    }
    if (!dgamma && !dbeta) return hipSuccess;
    hipLaunchKernelGGL(norm_fold_kernel, dim3((unsigned)min64((2 * a.D + 63) / 64, kMostGroups)), dim3(1024), 0, s, a.part, a.D, parts,
                       dgamma, dbeta);
    return hipGetLastError();
}

// f(type of X, type of Y) for the pairs of types that the operator takes: equal
// ones, and either type in fp32 beside the other in 16 bits.
template <typename F>
hipError_t with_types(int32_t x, int32_t y, F &&f) {
    if (x == ZI_F32 && y == ZI_F32) return f(float{}, float{});
    if (x == ZI_F32 && y == ZI_F16) return f(float{}, f16_t{});
    if (x == ZI_F32 && y == ZI_BF16) return f(float{}, bf16_t{});
    if (x == ZI_F16 && y == ZI_F16) return f(f16_t{}, f16_t{});
    if (x == ZI_F16 && y == ZI_F32) return f(f16_t{}, float{});
    if (x == ZI_BF16 && y == ZI_BF16) return f(bf16_t{}, bf16_t{});
    if (x == ZI_BF16 && y == ZI_F32) return f(bf16_t{}, float{});
    return hipErrorInvalidValue;
}

bool known(int32_t d) { return d == ZI_F16 || d == ZI_BF16 || d == ZI_F32; }
uint64_t size_of(int32_t d) { return d == ZI_F32 ? 4 : 2; }

zi_status check(const zi_norm *n, NormArgs *a) {
    if (!n) return fail(ZI_ERR_ARG, "norm is NULL");
    if (n->T < 0 || n->T > INT32_MAX) return fail(ZI_ERR_SHAPE, "T = %lld: 0 .. 2^31 - 1 rows", (long long)n->T);
    if (n->D < 1 || n->D > INT32_MAX) return fail(ZI_ERR_SHAPE, "D = %lld: 1 .. 2^31 - 1 columns", (long long)n->D);
    if (!known(n->x_dtype) || !known(n->y_dtype) || !known(n->p_dtype))
        return fail(ZI_ERR_ARG, "unknown dtype (x %d, y %d, p %d)", n->x_dtype, n->y_dtype, n->p_dtype);
    if (n->x_dtype != n->y_dtype && n->x_dtype != ZI_F32 && n->y_dtype != ZI_F32)
        return fail(ZI_ERR_ARG, "x_dtype and y_dtype are two different 16-bit types");
    if (!(n->eps >= 0.f) || !(n->eps < INFINITY)) return fail(ZI_ERR_ARG, "eps = %g", (double)n->eps);
    const int64_t ld[4] = {n->ldx, n->ldr, n->lds, n->ldy};
    for (int64_t l : ld)
        if (l != 0 && l < n->D) return fail(ZI_ERR_SHAPE, "a row stride of %lld is less than D", (long long)l);
    *a = NormArgs{};
    a->T = n->T;
    a->D = n->D;
    a->ldx = n->ldx ? n->ldx : n->D;
    a->ldr = n->ldr ? n->ldr : n->D;
    a->lds = n->lds ? n->lds : n->D;
    a->ldy = n->ldy ? n->ldy : n->D;
    a->eps = n->eps;
    a->width = (float)n->D;
    a->p_dtype = n->p_dtype;
    return ZI_OK;
}

bool aligned(const void *p, uint64_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

}  // namespace

extern "C" zi_status zi_layer_norm_fwd(const zi_norm *n, const void *X, const void *R, const void *gamma,
                                       const void *beta, void *S, void *Y, float *mean, float *rstd, void *stream) {
    clear_error();
    NormArgs a;
    zi_status st = check(n, &a);
    if (st != ZI_OK) return st;
    if (n->T == 0) return ZI_OK;
    if (!X || !Y) return fail(ZI_ERR_ARG, "X and Y are required");
    if (S && !R) return fail(ZI_ERR_ARG, "S is written with R only (without it, S is X)");
    const uint64_t xs = size_of(n->x_dtype), ys = size_of(n->y_dtype), ps = size_of(n->p_dtype);
    if (!aligned(X, xs) || !aligned(S, xs) || !aligned(R, ys) || !aligned(Y, ys) || !aligned(gamma, ps) ||
        !aligned(beta, ps) || !aligned(mean, 4) || !aligned(rstd, 4))
        return fail(ZI_ERR_ALIGN, "a pointer is not aligned to its element");
    a.X = X;
    a.R = R;
    a.S = S;
    a.Y = Y;
    a.gamma = gamma;
    a.beta = beta;
    a.mean = mean;
    a.rstd = rstd;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = with_types(n->x_dtype, n->y_dtype, [&](auto x, auto y) {
        return R ? run_fwd<decltype(x), decltype(y), true>(a, s) : run_fwd<decltype(x), decltype(y), false>(a, s);
    });
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "layer norm forward: %s", hipGetErrorString(e));
    return ZI_OK;
}

extern "C" uint64_t zi_layer_norm_bwd_bytes(int64_t T, int64_t D) {
    if (T < 0 || D < 1) return 0;
    // where wider rows take fewer parts, the room stays: a workspace for T rows of
    // D columns holds any fewer of both
    uint64_t most = 0;
    for (int64_t d : {min64(D, 4096), min64(D, 8192), D}) {
        const uint64_t sums = (uint64_t)min64(T, parts_of(d)) * 2 * (uint64_t)d;
        if (sums > most) most = sums;
    }
    return most * 4;
}

extern "C" zi_status zi_layer_norm_bwd(const zi_norm *n, const void *dY, const void *S, const void *gamma,
                                       const float *mean, const float *rstd, const void *dS, void *dX, float *dgamma,
                                       float *dbeta, void *workspace, uint64_t workspace_bytes, void *stream) {
    clear_error();
    NormArgs a;
    zi_status st = check(n, &a);
    if (st != ZI_OK) return st;
    if (n->T > 0 && (!dY || !S || !mean || !rstd || !dX))
        return fail(ZI_ERR_ARG, "dY, S, mean, rstd and dX are required");
    const uint64_t xs = size_of(n->x_dtype), ys = size_of(n->y_dtype), ps = size_of(n->p_dtype);
    if (!aligned(S, xs) || !aligned(dS, xs) || !aligned(dX, xs) || !aligned(dY, ys) || !aligned(gamma, ps) ||
        !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(dgamma, 4) || !aligned(dbeta, 4))
        return fail(ZI_ERR_ALIGN, "a pointer is not aligned to its element");
    const bool sums = dgamma || dbeta;
    if (sums && n->T > 0) {
        const uint64_t need = zi_layer_norm_bwd_bytes(n->T, n->D);
        if (!workspace || workspace_bytes < need)
            return fail(ZI_ERR_BUDGET, "the workspace holds %llu B, dgamma and dbeta need %llu",
                        (unsigned long long)(workspace ? workspace_bytes : 0), (unsigned long long)need);
        if (!aligned(workspace, 256)) return fail(ZI_ERR_ALIGN, "the workspace is not 256-byte aligned");
    }
    a.S = const_cast<void *>(S);
    a.Y = const_cast<void *>(dY);
    a.gamma = gamma;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dS = dS;
    a.dX = dX;
    a.part = sums ? static_cast<float *>(workspace) : nullptr;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = with_types(n->x_dtype, n->y_dtype, [&](auto x, auto y) {
        return run_bwd<decltype(x), decltype(y)>(a, dgamma, dbeta, s);
    });
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "layer norm backward: %s", hipGetErrorString(e));
    return ZI_OK;
}
