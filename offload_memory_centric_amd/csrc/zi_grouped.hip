// zi_grouped.hip -- products of many weights, each with a share of the rows: the
// experts of a mixture.  Group g has rows [offsets[g], offsets[g + 1]) of X and Y and
// the weight W_g (out-major, as the tiled linear's W^t):
//   forward  Y = X W_g^T, with GeLU A = X W_g^T, Y = GeLU(A)
//   dX       dX = dY W_g, with GeLU times GeLU'(A)
//   dW       dW_g (+)= dY_g^T X_g
// The offsets stay on the device: a workgroup finds its tile among all groups' by a
// scan, so that nothing waits for the host.  Most run on the MFMA kernel of zi_gemm.h,
// on macro-tiles of 256, 128 or 64 rows and columns; groups of a few rows, as in
// serving, which only wait for their weights, on the kernels here (forward and dX).
//
// Long reductions run at the matrix cores' rate under the card's power (32768 rows of
// 8 groups, 8192 x 32768 bf16, GeLU with both outputs: 12.8 ms, 1380 TFLOP/s).  With one
// macro-tile of 256 a compute unit nothing overlaps its epilogue, so shorter ones lose
// that share: dW of 16 groups, 32768 rows, 2048 x 8192 into fp32, 930 to 950 us, 1170
// TFLOP/s; dX with GeLU' of 24 groups, 14211 rows, 5000 x 2048 fp16, 371 to 385 us, 770
// TFLOP/s, of whose tiles a sixth are the groups' ragged ends.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "zi_grouped_choice.h"
#include "zi_host.h"
#include "zi_stream.h"

namespace zi {
namespace {

// The sums of the WAVES waves meet in LDS in a fixed order, and are stored: 16 QF columns
// from q0 of the rows from p0.
template <typename T, int EPI, int QF, int WAVES>
__device__ __forceinline__ void few_store(const GroupArgs &a, const GroupTile &gt, int64_t q0, int64_t p0, const f32x4 (&acc)[QF],
                                          char *lds) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    f32x4(*sums)[QF][64] = reinterpret_cast<f32x4(*)[QF][64]>(lds);
#pragma unroll
    for (int i = 0; i < QF; ++i) sums[wave][i][lane] = acc[i];
    __syncthreads();
    for (int t = tid; t < QF * 64; t += 64 * WAVES) {
        const int f = t >> 6, ln = t & 63;
        f32x4 v = sums[0][f][ln];
#pragma unroll
        for (int k = 1; k < WAVES; ++k) v += sums[k][f][ln];
        const int64_t q = q0 + 16 * f + 4 * (ln >> 4), p = p0 + (ln & 15);
        if (p >= gt.hi || q >= a.cols) continue;
        const int64_t off = p * a.ldc + q;
        if constexpr (EPI == EPI_F32) {
            *reinterpret_cast<f32x4 *>(static_cast<float *>(a.C) + off) = v;
        } else {
            if constexpr (EPI == EPI_DACT) {
                const u32x2 pre = *reinterpret_cast<const u32x2 *>(a.pre + p * a.ldpre + q);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] *= gelu_slope_f32(value16<T>((pre[e >> 1] >> (16 * (e & 1))) & 0xffffu));
            }
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

// 16 rows of one group by 32 columns.  The four waves share the reduction, each with
// a ring of its own in LDS, so that none waits for another before the end: steps of 64
// values, whose copies fetch whole lines of 128 bytes (chunks permuted as RcOperand's),
// three steps at a time, two workgroups a compute unit; rows past the group's are not
// fetched.  Bound by HBM, once W streams: 179 MB in 31.8 us are 5.6 TB/s.  (32 rows
// unevenly over 64 experts, 2048 x 1408 bf16: 33.4 us; with 64 columns and four steps,
// one workgroup a unit, 42.8; one row, 8192 x 8192: 26.4 and 28.8.)  Each workgroup begins
// at another step: where W's rows are a power of two apart, the same columns of all rows
// lie in few of the memory's channels.  The sums meet in LDS in a fixed order.
template <typename T, int EPI>
__global__ __launch_bounds__(256) void few_rows_kernel(GroupArgs a, int tiles_q) {
    constexpr int QF = 2, DEPTH = 3, STAGE = (16 * QF + 16) * 128, NC = 2 * QF + 2;
    __shared__ __attribute__((aligned(1024))) char lds[4 * DEPTH * STAGE];
    GroupTile gt;
    if (!find_group_tile<16>(a.offsets, a.groups, a.total, blockIdx.x, tiles_q, 64, gt)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4, row8 = lane >> 3;
    const int64_t q0 = (int64_t)gt.tq * (16 * QF), p0 = gt.lo + (int64_t)gt.tp * 16;
    const int group = __builtin_amdgcn_readfirstlane(gt.group);
    const rsrc_t wr = make_rsrc(reinterpret_cast<const char *>(static_cast<const uint16_t *>(a.Q) + group * a.q_group + q0 * a.ldq));
    const rsrc_t xr = make_rsrc(reinterpret_cast<const char *>(static_cast<const uint16_t *>(a.P) + p0 * a.ldp));
    const int red = (int)a.red, all = (red + 63) / 64;
    const int from = all * wave / 4, steps = all * (wave + 1) / 4 - from;
    const int turn = steps > 0 ? (int)(blockIdx.x * 5u % (unsigned)steps) : 0;
    const uint32_t at = lds_addr(lds) + (uint32_t)(wave * DEPTH * STAGE);
    // a copy is 8 rows of 128 bytes; its lane's chunk depends on the row's bit 3 alone
    uint32_t wo[2 * QF], xo[2], ck[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) ck[j] = (uint32_t)(((lane & 7) ^ (((8 * j + row8) >> 1) & 7)) * 8);
#pragma unroll
    for (int j = 0; j < 2 * QF; ++j) {
        const int row = 8 * j + row8;
        wo[j] = q0 + row < a.cols ? (uint32_t)((row * a.ldq + ck[j & 1]) * 2) : kOOB;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) xo[j] = p0 + 8 * j + row8 < gt.hi ? (uint32_t)(((8 * j + row8) * a.ldp + ck[j]) * 2) : kOOB;
    uint32_t fo[2];  // this lane's fragment of the two halves of a step, within 16 rows
#pragma unroll
    for (int h = 0; h < 2; ++h) fo[h] = (uint32_t)(c * 128 + (((4 * h + g) ^ ((c >> 1) & 7)) << 4));

    auto issue = [&](int s) __attribute__((always_inline)) {  // past the last step: zeros
        const uint32_t stage = at + (uint32_t)(s % DEPTH) * STAGE;
        const int turned = s + turn < steps ? s + turn : s + turn - steps;
        const uint32_t k0 = s < steps ? (uint32_t)(from + turned) * 64 : (uint32_t)red;
        const uint32_t left = (uint32_t)red - k0;
        const uint32_t k2[2] = {ck[0] < left ? k0 * 2 : kOOB, ck[1] < left ? k0 * 2 : kOOB};
        // (two offsets past the descriptor's range stay past it when added)
#pragma unroll
        for (int j = 0; j < 2 * QF; ++j) copy16(wr, stage + j * 1024, wo[j] + k2[j & 1]);
#pragma unroll
        for (int j = 0; j < 2; ++j) copy16(xr, stage + QF * 2048 + j * 1024, xo[j] + k2[j]);
    };
    f32x4 acc[QF] = {};
#pragma unroll
    for (int s = 0; s < DEPTH - 1; ++s) issue(s);
    for (int s = 0; s < steps; ++s) {
        // step s has landed, and step s - 1 has been read
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((DEPTH - 2) * NC) : "memory");
        issue(s + DEPTH - 1);
        const uint32_t stage = at + (uint32_t)(s % DEPTH) * STAGE;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4 x =
                *reinterpret_cast<const __attribute__((address_space(3))) u32x4 *>((uintptr_t)(stage + QF * 2048 + fo[h]));
#pragma unroll
            for (int i = 0; i < QF; ++i)
                acc[i] = mfma<T>(*reinterpret_cast<const __attribute__((address_space(3))) u32x4 *>((uintptr_t)(stage + i * 2048 + fo[h])),
                                 x, acc[i]);
        }
    }
    // every copy has landed and every read returned before the rings hold the sums
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    few_store<T, EPI, QF, 4>(a, gt, q0, p0, acc, lds);
}

// dX of a few rows: 16 rows of one group by 32 columns, whose eight waves share the
// reduction over W's rows, each with a ring of its own of chunks of 32 of them: 64 bytes
// of each, read back across the rows (ds_read_b64_tr_b16), and the same values of dY's
// rows.  Bound by what one workgroup's 120 KB in flight fetch where tiles are few, which
// a macro-tile of 64 takes longer over.  (21 rows of 2 groups, 22488 -> 160 bf16: 46 us,
// 146 with tiles of 64.)
template <typename T, int EPI>
__global__ __launch_bounds__(512) void few_rows_dx_kernel(GroupArgs a, int tiles_q) {
    constexpr int QF = 2, DEPTH = 6, kChunk = 32, WB = kChunk * 64, STAGE = WB + 16 * 64, NC = 3;
    __shared__ __attribute__((aligned(1024))) char lds[8 * DEPTH * STAGE];
    GroupTile gt;
    if (!find_group_tile<16>(a.offsets, a.groups, a.total, blockIdx.x, tiles_q, 32, gt)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4, row16 = lane >> 2, piece = (lane & 3) * 8;
    const int64_t q0 = (int64_t)gt.tq * (16 * QF), p0 = gt.lo + (int64_t)gt.tp * 16;
    const int group = __builtin_amdgcn_readfirstlane(gt.group);
    const uint16_t *W = static_cast<const uint16_t *>(a.Q) + group * a.q_group + q0;
    const rsrc_t yr = make_rsrc(reinterpret_cast<const char *>(static_cast<const uint16_t *>(a.P) + p0 * a.ldp));
    const int red = (int)a.red, all = (red + kChunk - 1) / kChunk;
    const int from = all * wave / 8, steps = all * (wave + 1) / 8 - from;
    const int turn = steps > 0 ? (int)(blockIdx.x * 5u % (unsigned)steps) : 0;
    const uint32_t at = lds_addr(lds) + (uint32_t)(wave * DEPTH * STAGE);
    // a copy is 16 rows of 64 bytes
    const uint32_t wo = q0 + piece < a.cols ? (uint32_t)((row16 * a.ldq + piece) * 2) : kOOB, w16 = (uint32_t)(32 * a.ldq);
    const uint32_t yo = p0 + row16 < gt.hi ? (uint32_t)((row16 * a.ldp + piece) * 2) : kOOB;
    const uint32_t fw = (uint32_t)((8 * g + (c >> 2)) * 64 + 8 * (c & 3)), fy = (uint32_t)(WB + c * 64 + 16 * g);

    auto issue = [&](int s) __attribute__((always_inline)) {  // past the last step: zeros
        const uint32_t stage = at + (uint32_t)(s % DEPTH) * STAGE;
        const int turned = s + turn < steps ? s + turn : s + turn - steps;
        const int m0 = s < steps ? (from + turned) * kChunk : 0, left = s < steps ? red - m0 : 0;
        const rsrc_t wr = make_rsrc(reinterpret_cast<const char *>(W + m0 * a.ldq));
        copy16(wr, stage, row16 < left ? wo : kOOB);
        copy16(wr, stage + 1024, 16 + row16 < left ? wo + w16 : kOOB);
        copy16(yr, stage + WB, piece < left ? yo + (uint32_t)(m0 * 2) : kOOB);
    };
    f32x4 acc[QF] = {};
#pragma unroll
    for (int s = 0; s < DEPTH - 1; ++s) issue(s);
    for (int s = 0; s < steps; ++s) {
        // step s has landed, and step s - 1 has been read
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((DEPTH - 2) * NC) : "memory");
        issue(s + DEPTH - 1);
        const uint32_t stage = at + (uint32_t)(s % DEPTH) * STAGE;
        const u32x4 y = *reinterpret_cast<const __attribute__((address_space(3))) u32x4 *>((uintptr_t)(stage + fy));
#pragma unroll
        for (int i = 0; i < QF; ++i) {
            const u32x2 w0 = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                           (__attribute__((address_space(3))) s16x4 *)(uintptr_t)(stage + fw + 32 * i)));
            const u32x2 w1 = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                           (__attribute__((address_space(3))) s16x4 *)(uintptr_t)(stage + fw + 32 * i + 256)));
            acc[i] = mfma<T>(u32x4{w0[0], w0[1], w1[0], w1[1]}, y, acc[i]);
        }
    }
    // every copy has landed and every read returned before the rings hold the sums
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier\n\ts_nop 7\n\ts_nop 7" ::: "memory");
    few_store<T, EPI, QF, 8>(a, gt, q0, p0, acc, lds);
}

template <typename T, int EPI>
hipError_t run_few(const GroupArgs &a, hipStream_t s) {
    const int64_t grid = row_grid(a.total, a.groups, a.cols, 16, 32);
    hipLaunchKernelGGL((few_rows_kernel<T, EPI>), dim3((unsigned)grid), dim3(256), 0, s, a, (int)ceil_div(a.cols, 32));
    return hipGetLastError();
}
template <typename T, int EPI>
hipError_t run_few_dx(const GroupArgs &a, hipStream_t s) {
    const int64_t grid = row_grid(a.total, a.groups, a.cols, 16, 32);
    hipLaunchKernelGGL((few_rows_dx_kernel<T, EPI>), dim3((unsigned)grid), dim3(512), 0, s, a, (int)ceil_div(a.cols, 32));
    return hipGetLastError();
}
template <typename T>
hipError_t few_dx(const GroupArgs &a, hipStream_t s) {
    if (a.pre) return run_few_dx<T, EPI_DACT>(a, s);
    return a.out_f32 ? run_few_dx<T, EPI_F32>(a, s) : run_few_dx<T, EPI_LP>(a, s);
}
template <typename T>
hipError_t few(const GroupArgs &a, hipStream_t s) {
    if (a.act) return run_few<T, EPI_ACT>(a, s);
    return a.out_f32 ? run_few<T, EPI_F32>(a, s) : run_few<T, EPI_LP>(a, s);
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

zi_status too_many_tiles(const zi_grouped *g) {
    return fail(ZI_ERR_SHAPE, "R = %lld, K = %lld, M = %lld, E = %d: more than 2^23 - 8 tiles of 256 x 256", (long long)g->R,
                (long long)g->K, (long long)g->M, g->E);
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
    const int tile = grouped_fwd_tile(g->R, g->K, g->M, g->E);
    if (!tile) return too_many_tiles(g);
    hipError_t e;
    if (tile == kFewRows)
        e = g->dtype == ZI_F16 ? few<_Float16>(a, s) : few<__bf16>(a, s);
    else
        e = launch_grouped_fwd(g->dtype, tile, a, s);
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
    const int tile = grouped_dx_tile(g->R, g->K, g->M, g->E);
    if (!tile) return too_many_tiles(g);
    hipError_t e;
    if (tile == kFewRows)
        e = g->dtype == ZI_F16 ? few_dx<_Float16>(a, s) : few_dx<__bf16>(a, s);
    else
        e = launch_grouped_dx(g->dtype, tile, a, s);
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
    const int tile = grouped_dw_tile(g->R, g->K, g->M, g->E, g->accumulate != 0);
    if (!tile) return too_many_tiles(g);
    const hipError_t e = launch_grouped_dw(g->dtype, tile, a, s);
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "grouped weight gradient: %s", hipGetErrorString(e));
    return ZI_OK;
}
