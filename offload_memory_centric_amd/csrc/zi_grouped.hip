// zi_grouped.hip -- products of many weights, each with a share of the rows: the
// experts of a mixture.  Group g has rows [offsets[g], offsets[g + 1]) of X and Y and
// the weight W_g (out-major, as the tiled linear's W^t):
//   forward  Y = X W_g^T, with GeLU A = X W_g^T, Y = GeLU(A)
//   dX       dX = dY W_g, with GeLU times GeLU'(A)
//   dW       dW_g (+)= dY_g^T X_g
// The offsets stay on the device: a workgroup finds its tile among all groups' by a
// scan, so that nothing waits for the host.  Groups of many rows run on the MFMA
// kernel of zi_gemm.h (256, 128 or 64 rows and columns a workgroup).  Groups of a few
// rows, as in serving, only wait for their weights: the kernel here streams W from
// memory into the matrix cores' registers, past LDS.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdlib.h>
#include <stdint.h>

#include "zi_gemm.h"
#include "zi_host.h"
#include "zi_stream.h"

namespace zi {
namespace {

// 16 PF rows of one group by 16 QF columns: four waves share the reduction, each in
// steps of 32 (stream_product); the sums meet in LDS in a fixed order.
template <typename T, int QF, int PF, int EPI>
__global__ __launch_bounds__(256) void few_rows_kernel(GroupArgs a, int tiles_q) {
    constexpr int kAhead = PF == 4 ? 2 : 4;
    __shared__ f32x4 sums[4][QF * PF][64];
    GroupTile gt;
    if (!find_group_tile<16 * PF>(a.offsets, a.groups, a.total, blockIdx.x, tiles_q, 64, gt)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t q0 = (int64_t)gt.tq * (16 * QF), p0 = gt.lo + (int64_t)gt.tp * (16 * PF);
    const int group = __builtin_amdgcn_readfirstlane(gt.group);
    uint32_t wo[QF], xo[PF];
    fragment_offsets(a.cols - q0, a.ldq, wo);
    fragment_offsets(gt.hi - p0, a.ldp, xo);
    const int red = (int)a.red, steps = (red + 31) / 32, share = (steps + 3) / 4;
    f32x4 acc[QF][PF] = {};
    stream_product<T, QF, PF, kAhead>(buffer_of(static_cast<const uint16_t *>(a.Q) + group * a.q_group + q0 * a.ldq), wo,
                                      buffer_of(static_cast<const uint16_t *>(a.P) + p0 * a.ldp), xo, wave * share,
                                      min((wave + 1) * share, steps), red, acc);
#pragma unroll
    for (int i = 0; i < QF; ++i)
#pragma unroll
        for (int j = 0; j < PF; ++j) sums[wave][i * PF + j][lane] = acc[i][j];
    __syncthreads();
    for (int t = tid; t < QF * PF * 64; t += 256) {
        const int f = t >> 6, ln = t & 63;
        f32x4 v = sums[0][f][ln];
#pragma unroll
        for (int k = 1; k < 4; ++k) v += sums[k][f][ln];
        const int64_t q = q0 + 16 * (f / PF) + 4 * (ln >> 4), p = p0 + 16 * (f % PF) + (ln & 15);
        if (p >= gt.hi || q >= a.cols) continue;
        const int64_t off = p * a.ldc + q;
        if constexpr (EPI == EPI_F32) {
            *reinterpret_cast<f32x4 *>(static_cast<float *>(a.C) + off) = v;
        } else {
            uint32_t b[4], h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                b[e] = bits16<T>(v[e]);
                h[e] = EPI == EPI_ACT ? bits16<T>(gelu_f32(v[e])) : b[e];
            }
            *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.C) + off) = u32x2{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
            if (EPI == EPI_ACT && a.C2)
                *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.C2) + p * a.ldpre + q) =
                    u32x2{b[0] | (b[1] << 16), b[2] | (b[3] << 16)};
        }
    }
}

int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
int64_t min64(int64_t x, int64_t y) { return x < y ? x : y; }

template <typename T, int QF, int PF, int EPI>
hipError_t run_few(const GroupArgs &a, hipStream_t s) {
    const int64_t tiles_q = ceil_div(a.cols, 16 * QF);
    const int64_t rows = a.total / (16 * PF) + min64(a.groups, a.total);
    const int64_t grid = ceil_div(rows * tiles_q, 8) * 8;
    if (grid > INT32_MAX / 256) return hipErrorInvalidValue;
    hipLaunchKernelGGL((few_rows_kernel<T, QF, PF, EPI>), dim3((unsigned)grid), dim3(256), 0, s, a, (int)tiles_q);
    return hipGetLastError();
}
// 64 columns a workgroup; 16 where that leaves compute units without one.
template <typename T, int EPI>
hipError_t few_sized(const GroupArgs &a, int pf, hipStream_t s) {
    const bool narrow = min64(a.groups, a.total) * ceil_div(a.cols, 64) < 256;
    if (pf == 1) return narrow ? run_few<T, 1, 1, EPI>(a, s) : run_few<T, 4, 1, EPI>(a, s);
    if (pf == 2) return narrow ? run_few<T, 1, 2, EPI>(a, s) : run_few<T, 4, 2, EPI>(a, s);
    return narrow ? run_few<T, 1, 4, EPI>(a, s) : run_few<T, 4, 4, EPI>(a, s);
}
template <typename T>
hipError_t few(const GroupArgs &a, int pf, hipStream_t s) {
    if (a.act) return few_sized<T, EPI_ACT>(a, pf, s);
    return a.out_f32 ? few_sized<T, EPI_F32>(a, pf, s) : few_sized<T, EPI_LP>(a, pf, s);
}

// The macro-tile that takes least, by rounds of workgroups on 256 compute units: a
// round of tiles of 256 (one a unit) counts 1, of 128 (two a unit) 0.71, of 64 (four)
// 0.62, from what a unit multiplies in each.  `groups` of the row tiles are half full.
int tile_of(int64_t rows, int64_t cols, int64_t groups, bool ragged) {
    if (getenv("GT")) return atoi(getenv("GT"));
    int best = 256;
    double least = 0;
    for (int tile = 256, each = 1; tile >= 64; tile /= 2, each *= 2) {
        const double row_tiles = ragged ? (double)rows / tile + 0.5 * (double)groups : (double)ceil_div(rows, tile) * (double)groups;
        const double rounds = ceil(row_tiles * (double)ceil_div(cols, tile) / (256.0 * each));
        const double t = rounds * (tile == 256 ? 1.0 : tile == 128 ? 0.71 : 0.62);
        if (least == 0 || t < least) {
            best = tile;
            least = t;
        }
    }
    return best;
}

bool aligned(const void *p, uint64_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

zi_status check(const zi_grouped *g) {
    if (!g) return fail(ZI_ERR_ARG, "grouped is NULL");
    if (g->R < 0 || g->R > ((int64_t)1 << 30)) return fail(ZI_ERR_SHAPE, "R = %lld: 0 .. 2^30 rows", (long long)g->R);
    if (g->E < 1 || g->E > ZI_GROUPS_MOST) return fail(ZI_ERR_SHAPE, "E = %d: 1 .. %d groups", g->E, ZI_GROUPS_MOST);
    if (g->K < 8 || g->M < 8 || g->K % 8 || g->M % 8 || g->K > kGroupLd || g->M > kGroupLd)
        return fail(ZI_ERR_SHAPE, "K = %lld, M = %lld: multiples of 8 up to 2^20", (long long)g->K, (long long)g->M);
    const int64_t lds[4] = {g->ldx, g->ldy, g->lda, g->ldw};
    for (int64_t ld : lds)
        if (ld < 0 || ld % 8 || ld > kGroupLd) return fail(ZI_ERR_SHAPE, "row strides are multiples of 8 up to 2^20");
    if ((g->ldx && g->ldx < g->K) || (g->ldw && g->ldw < g->K) || (g->ldy && g->ldy < g->M))
        return fail(ZI_ERR_SHAPE, "a row stride is less than a row");
    const int64_t ldw = g->ldw ? g->ldw : g->K;
    if (g->ldg && (g->ldg % 8 || g->ldg < (g->M - 1) * ldw + g->K)) return fail(ZI_ERR_SHAPE, "the groups' weights overlap or are not aligned");
    if (g->dtype != ZI_F16 && g->dtype != ZI_BF16) return fail(ZI_ERR_ARG, "dtype %d: fp16 or bf16", g->dtype);
    if (g->out_dtype != g->dtype && g->out_dtype != ZI_F32) return fail(ZI_ERR_ARG, "out_dtype %d: dtype or fp32", g->out_dtype);
    return ZI_OK;
}

// What the products share.
GroupArgs args_of(const zi_grouped *g, const int32_t *offsets) {
    GroupArgs a = {};
    a.offsets = offsets;
    a.groups = g->E;
    a.total = g->R;
    a.out_f32 = g->out_dtype == ZI_F32;
    const int64_t ldw = g->ldw ? g->ldw : g->K;
    a.q_group = a.c_group = g->ldg ? g->ldg : g->M * ldw;
    return a;
}

}  // namespace
}  // namespace zi

using namespace zi;

extern "C" zi_status zi_grouped_fwd(const zi_grouped *g, const void *X, const void *W, const int32_t *offsets, void *Y, void *A,
                                    void *stream) {
    clear_error();
    const zi_status st = check(g);
    if (st != ZI_OK) return st;
    if (A && !g->gelu) return fail(ZI_ERR_ARG, "A is the input of GeLU, which is not asked for");
    if (g->gelu && g->out_dtype == ZI_F32) return fail(ZI_ERR_ARG, "with GeLU the output has the operands' type");
    if (A && g->lda && g->lda < g->M) return fail(ZI_ERR_SHAPE, "A's row stride is less than M");
    if (g->R == 0) return ZI_OK;
    if (!X || !W || !offsets || !Y) return fail(ZI_ERR_ARG, "X, W, offsets and Y are required");
    if (!aligned(X, 16) || !aligned(W, 16) || !aligned(Y, 16) || !aligned(A, 16) || !aligned(offsets, 4))
        return fail(ZI_ERR_ALIGN, "a matrix is not 16-byte aligned, or offsets not to their element");
    GroupArgs a = args_of(g, offsets);
    a.Q = W;
    a.ldq = g->ldw ? g->ldw : g->K;
    a.P = X;
    a.ldp = g->ldx ? g->ldx : g->K;
    a.C = Y;
    a.ldc = g->ldy ? g->ldy : g->M;
    a.act = g->gelu;
    a.C2 = A;
    a.ldpre = g->lda ? g->lda : g->M;
    a.rows = g->R;
    a.cols = g->M;
    a.red = g->K;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t live = min64(g->E, g->R);
    // rows of an average group with any: up to 32 the weights' bytes are what counts
    const int64_t mean = ceil_div(g->R, live);
    hipError_t e;
    if (getenv("PF") ? atoi(getenv("PF")) > 0 : mean <= 32) {
        const int pf = getenv("PF") ? atoi(getenv("PF")) : mean <= 8 ? 1 : mean <= 16 ? 2 : 4;
        e = g->dtype == ZI_F16 ? few<_Float16>(a, pf, s) : few<__bf16>(a, pf, s);
    } else {
        e = launch_grouped_fwd(g->dtype, tile_of(g->R, g->M, live, true), a, s);
    }
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "grouped forward: %s", hipGetErrorString(e));
    return ZI_OK;
}

extern "C" zi_status zi_grouped_dx(const zi_grouped *g, const void *dY, const void *W, const int32_t *offsets, const void *A,
                                   void *dX, void *stream) {
    clear_error();
    const zi_status st = check(g);
    if (st != ZI_OK) return st;
    if (A && g->out_dtype == ZI_F32) return fail(ZI_ERR_ARG, "with A the output has the operands' type");
    if (A && g->lda && g->lda < g->K) return fail(ZI_ERR_SHAPE, "A's row stride is less than K");
    if (g->R == 0) return ZI_OK;
    if (!dY || !W || !offsets || !dX) return fail(ZI_ERR_ARG, "dY, W, offsets and dX are required");
    if (!aligned(dY, 16) || !aligned(W, 16) || !aligned(dX, 16) || !aligned(A, 16) || !aligned(offsets, 4))
        return fail(ZI_ERR_ALIGN, "a matrix is not 16-byte aligned, or offsets not to their element");
    GroupArgs a = args_of(g, offsets);
    a.Q = W;
    a.ldq = g->ldw ? g->ldw : g->K;
    a.P = dY;
    a.ldp = g->ldy ? g->ldy : g->M;
    a.C = dX;
    a.ldc = g->ldx ? g->ldx : g->K;
    a.pre = static_cast<const uint16_t *>(A);
    a.ldpre = g->lda ? g->lda : g->K;
    a.rows = g->R;
    a.cols = g->K;
    a.red = g->M;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = launch_grouped_dx(g->dtype, tile_of(g->R, g->K, min64(g->E, g->R), true), a, s);
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "grouped input gradient: %s", hipGetErrorString(e));
    return ZI_OK;
}

extern "C" zi_status zi_grouped_dw(const zi_grouped *g, const void *X, const void *dY, const int32_t *offsets, void *dW,
                                   void *stream) {
    clear_error();
    const zi_status st = check(g);
    if (st != ZI_OK) return st;
    if (g->accumulate && g->out_dtype != ZI_F32) return fail(ZI_ERR_ARG, "only an fp32 gradient is accumulated");
    if (!offsets || !dW || (g->R > 0 && (!X || !dY))) return fail(ZI_ERR_ARG, "X, dY, offsets and dW are required");
    if (!aligned(X, 16) || !aligned(dY, 16) || !aligned(dW, 16) || !aligned(offsets, 4))
        return fail(ZI_ERR_ALIGN, "a matrix is not 16-byte aligned, or offsets not to their element");
    if (g->R == 0 && g->accumulate) return ZI_OK;
    GroupArgs a = args_of(g, offsets);
    a.Q = X;
    a.ldq = g->ldx ? g->ldx : g->K;
    a.P = dY;
    a.ldp = g->ldy ? g->ldy : g->M;
    a.C = dW;
    a.ldc = g->ldw ? g->ldw : g->K;
    a.rows = g->M;
    a.cols = g->K;
    a.red = g->R;
    a.accumulate = g->accumulate;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = launch_grouped_dw(g->dtype, tile_of(g->M, g->K, g->E, false), a, s);
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "grouped weight gradient: %s", hipGetErrorString(e));
    return ZI_OK;
}
