// zi_internal.h -- declarations shared by the library's own translation units
// (host API, ring model, kernels).  Not installed; the public ABI is zi.h.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace zi {

// Which product a GEMM launch forms.  The output C[p][q] is row-major with q
// contiguous; "Q" is the operand indexed by q, "P" the operand indexed by p.
enum class GemmOp : int {
    Fwd = 0,      // Y_i[t][m]  = sum_k X[t][k] W^t_i[m][k]      (Q = W slot, P = X)
    FwdGelu = 1,  // same product; stores A = RNE(acc) (fp32 acc with out_f32) and H = RNE(GeLU(RNE(acc)))
    Dx = 2,       // dX[t][k]  (+)= sum_r dY[t][i*n+r] W^t_i[r][k] (Q = W slot^T, P = dY)
    Dw = 3,       // dW^t_i[m][k] = sum_t dY[t][i*n+m] X[t][k]    (Q = X^T,      P = dY^T)
};

struct GemmArgs {
    const void *Q;  // 16-bit elements
    int64_t ldq;
    const void *P;  // 16-bit elements
    int64_t ldp;
    void *C;        // output: 16-bit, or fp32 when out_f32 / Dx
    int64_t ldc;
    void *C2;       // FwdGelu: H output (same layout as C)
    int64_t rows;   // extent of p
    int64_t cols;   // extent of q (multiple of 8)
    int64_t red;    // reduction length
    int accumulate; // Dx only: 0 = overwrite, 1 = add into C
    int out_f32;    // Fwd / Dw: write fp32 instead of the 16-bit format; FwdGelu: A in fp32
    // Two weight tiles held in different ring slots, consumed by one launch.
    // Dx: reduction rows k >= qsplit of Q come from Q2 (row k - qsplit);
    // qsplit a multiple of the kernel's step (64).  Fwd: output columns
    // q >= qsplit come from Q2 (row q - qsplit); qsplit a multiple of the
    // launch's macro-tile width (gemm_tile).  Q2 = null: no split.
    const void *Q2;
    int64_t qsplit;
    // Dx: at most this many workgroups (a multiple of 8), each taking several
    // output tiles in turn, the next tile's first copies and C loads issued
    // under the finished tile's stores; 0 = one workgroup per output tile.
    int32_t wg_cap;
    // FwdGelu: fp32 half-sums and arrival counters (workspace of
    // kSplitBytes, counters zero between launches) for splitting the
    // reduction of the launch's last, partial round of tiles between two
    // workgroups each, when at most half of split_cap (the workgroups that run
    // at once) would be busy in it; null: no split.  split_tail is set by the
    // launch: the number of such tiles.
    float *split_part;
    uint32_t *split_cnt;
    int32_t split_cap;
    int32_t split_tail;
};

// dtype: 1 = fp16, 2 = bf16.  Returns the launch status (hipGetLastError).
hipError_t launch_gemm(GemmOp op, int dtype, const GemmArgs &a, hipStream_t stream);

// A step x <- a x + (b A + c A^2) x, A = x x^T, of the orthogonalised update
// (zi_orth.hip).  Matrices are kept with their diagonals apart: A = D + O, with
// D in fp32 and O (zero on the diagonal) in fp16 as an operand and in fp32 for
// the linear term; likewise bA + cA^2 = diag(bd) + B.
//   Gram   acc = x x^T        D, O (C: fp16, o32: fp32 on and below the diagonal)
//   Poly   acc = O O          bd, B (C: fp16)
//   Apply  acc = B x          a x + bd x + acc (hi, lo: two fp16 planes), or `out` after the last step
// The first two are symmetric: tiles on and below the diagonal are formed, and
// those below it written on both sides.
enum class OrthOp : int { Gram = 0, Poly = 1, Apply = 2 };
struct OrthArgs : GemmArgs {
    int32_t pieces;       // workgroups that share the reduction of each of the last split_tail tiles
    const float *scale;   // Gram: x = *scale times its planes; Apply: the result is *scale times what they give
    float ca, cb, cc;     // a, b, c
    float *o32;           // [rows][ldc], as O
    float *diag, *bdiag;  // D, bd
    const uint16_t *hi;   // Apply: the planes of x, [rows][ldc]
    uint16_t *lo;
    int32_t diag_x;       // bd multiplies both planes; else hi alone, as B does
    uint16_t *hi_out;     // the new planes (lo is replaced in place); null: write `out`
    uint16_t *out;        // bf16
    int64_t out_p, out_q, out_ld;  // its extents along p and q, and its row stride
    int32_t out_t;                 // it is stored transposed: element (p, q) at out[q * out_ld + p]
};

// One of the products, on tiles of 256, 128 or 64 rows and columns.  rows, cols
// and red are multiples of 64.  split_part holds orth_split_bytes(tile) and
// split_cnt kOrthSplits counters, zero between launches.
hipError_t launch_orth(OrthOp op, int tile, const OrthArgs &a, hipStream_t stream);

// Workgroups that share tiles whose reduction is split: at most as many as run at
// once, one a compute unit with tiles of 256, two with 128, four with 64.
constexpr int kOrthUnits = 256;
constexpr int kOrthSplits = 4 * kOrthUnits;
constexpr uint64_t orth_split_bytes(int tile) { return (uint64_t)kOrthUnits * (256 / tile) * tile * tile * 4; }

// Workgroups (one macro-tile each) that launch_gemm runs for a product with
// `rows` output rows and `cols` output columns: the macro-tile is 256 x 256,
// or 192 x 320 / 320 x 192 (rows x columns) where that tile covers a forward's
// columns or a gradient's rows with clearly less padding.
int64_t gemm_workgroups(GemmOp op, int64_t rows, int64_t cols);
// That macro-tile: output rows and columns of one workgroup.
void gemm_tile(GemmOp op, int64_t rows, int64_t cols, int *tile_rows, int *tile_cols);

// Builds the per-device tables H = RNE16(GeLU(A)) over every 16-bit A (fp16
// and bf16) that the forward GeLU epilogue reads; enqueued on `stream`.
hipError_t build_gelu_tables(hipStream_t stream);

// dA[i] = RNE(dH[i] * GeLU'(A[i])), i < count; with out_f32 the fp32 product
// itself (dA then holds fp32 elements).
hipError_t launch_gelu_bwd(int dtype, const float *dH, const void *A, void *dA, int64_t count,
                           bool out_f32, hipStream_t stream);

// Reduction values per pipeline step of the GEMM kernels.
constexpr int kGemmStep = 64;

// Split GeLU forward: at most kSplitTiles tiles, each two fp32 half-sums of
// 256 x 256 (256 KiB), then one 32-bit counter per tile.
constexpr int kSplitTiles = 128;
constexpr uint64_t kSplitPartBytes = (uint64_t)kSplitTiles * 2 * 256 * 256 * 4;
constexpr uint64_t kSplitBytes = kSplitPartBytes + 512;

}  // namespace zi
