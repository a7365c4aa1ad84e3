// zi_grouped.hip -- products of many weights, each with a share of the rows: the
// experts of a mixture.  Group g has rows [offsets[g], offsets[g + 1]) of X and Y and
// the weight W_g (out-major, as the tiled linear's W^t):
//   forward  Y = X W_g^T, with GeLU A = X W_g^T, Y = GeLU(A)
//   dX       dX = dY W_g, with GeLU times GeLU'(A)
//   dW       dW_g (+)= dY_g^T X_g
// The offsets stay on the device: a workgroup finds its tile among all groups' by a
// scan, so that nothing waits for the host.  All run on the MFMA kernel of zi_gemm.h,
// on macro-tiles of 256, 128 or 64 rows and columns.  (Groups of a few rows, as in
// serving, only wait for their weights.  A kernel that read W from memory into the
// matrix cores' registers, 16 rows by 64 bytes at a time, took 33.9 us for 32 rows of
// 64 experts, 2048 x 1408 bf16; tiles of 64, whose copies into LDS fetch whole lines of
// 128 bytes, 26.5.)
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "zi_host.h"
#include "zi_internal.h"

namespace zi {
namespace {

int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
int64_t min64(int64_t x, int64_t y) { return x < y ? x : y; }

// The macro-tile that takes least, by its rounds of workgroups on 256 compute units, of
// which each holds one tile of 256, two of 128 or four of 64.  A round takes what the
// products of many shapes measured (us for a reduction of r thousand): 19.1 r + 14,
// 12.6 r + 6 and 12 r + 5; a tile that has its unit to itself 16.5 r + 14, 7.4 r + 5 and
// 6.2 r + 4.  Of a ragged operand's row tiles one a group is taken as half full.  (Over
// 45 products of 1 to 64 groups the choice is 1.5 % slower than the best tile on
// average; 20000 rows of 16 groups, 1024 x 1024: 74.0, 60.8 and 83.7 us forward.)
int tile_of(int64_t rows, int64_t cols, int64_t groups, double red, bool ragged) {
    const double r = red / 1000;
    int best = 256;
    double least = 0;
    for (int tile = 256; tile >= 64; tile /= 2) {
        const double row_tiles = ragged ? (double)rows / tile + 0.5 * (double)groups : (double)ceil_div(rows, tile) * (double)groups;
        const double each = row_tiles * (double)ceil_div(cols, tile) / 256;  // tiles a compute unit
        double t;
        if (tile == 256) {
            t = each > 1 ? ceil(each - 0.05) * (19.1 * r + 14) : 16.5 * r + 14;
        } else if (tile == 128) {
            t = each > 1 ? fmax(1, ceil(each / 2 - 0.05)) * (12.6 * r + 6) : 7.4 * r + 5;
        } else {
            const double alone = 6.2 * r + 4, full = 12 * r + 5;
            t = each > 4 ? each / 4 * full : alone + (full - alone) * fmax(0, each - 1) / 3;
        }
        if (least == 0 || t < 0.93 * least) {  // (where they are close, the larger)
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
    const hipError_t e = launch_grouped_fwd(g->dtype, tile_of(g->R, g->M, min64(g->E, g->R), (double)g->K, true), a, s);
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
    const hipError_t e = launch_grouped_dx(g->dtype, tile_of(g->R, g->K, min64(g->E, g->R), (double)g->M, true), a, s);
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
    const hipError_t e = launch_grouped_dw(g->dtype, tile_of(g->M, g->K, g->E, (double)g->R / g->E, false), a, s);
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "grouped weight gradient: %s", hipGetErrorString(e));
    return ZI_OK;
}
