// zi_adapter.hip -- low-rank adapters of many requests beside a shared projection.
//
// The T rows of a batch lie in S segments (a request's prompt, or its one new token),
// each with one of N adapters: A_n [r x K], B_n [r x M], the rank outermost in both.
//   U = A_n X^T (r x T, fp32),  Y = Y0 + s_n U^T B_n
// and backward, with dU = s_n B_n dY^T,
//   dX = dX0 + dU^T A_n,  dA_n = sum dU X,  dB_n = s_n sum U dY  over the adapter's rows.
// With the rank outermost everywhere these are three kernels:
//   shrink  U from X and A, dU from dY and B      reads the wide rows once
//   expand  Y from U and B, dX from dU and A      reads and writes the wide rows once
//   grad    dA from dU and X, dB from U and dY    reads the wide rows once
// All are bound by the bytes of the wide rows while r is small.  U is kept in fp32; where it
// is multiplied it is split into planes of the other operand's 16 bits, which the 16-bit
// matrix instruction takes at sixteen times the rate of the fp32 one.  Three of bf16 hold all
// 24 of its bits.  Two of fp16 hold 22 of those values that are no less than 2^-17 of the
// largest that shares their scale (a row's ranks in expand, 32 rows of a rank in grad), and
// smaller ones to within 2^-39 of that largest.  shrink's operands are 16-bit inputs,
// multiplied exactly.
// (20011 fp16 rows of 8192 by 8192 with r = 16: shrink 77 us, 4.3 TB/s, its parts' sum 5,
// expand 131, 5.0 TB/s.  Backward of 32768 bf16 rows, r = 32, dX in fp32: shrink 102 us,
// 5.2 TB/s, expand 405, 5.3 TB/s, grad for both 237, 4.5 TB/s.)
//
// A row's result depends on that row and its adapter alone: segments are multiplied one
// by one, so that an infinity or a NaN in one request or adapter reaches no other.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "zi_host.h"
#include "zi_stream.h"
#include "zi_vec.h"

namespace zi {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }
int64_t max64(int64_t a, int64_t b) { return a > b ? a : b; }
uint64_t round_up(uint64_t n) { return (n + 255) / 256 * 256; }

struct Segments {
    const int32_t *offsets;  // [count + 1]
    const int32_t *ids;      // [count]
    int32_t count, adapters, rows;
};

// f(n, a, b) for the runs [a, b) of rows, in order and without gaps, that cover
// [b0, b1): n is the adapter of the run, -1 where there is none.  Whatever the offsets
// hold, every row comes once.
template <typename F>
__device__ __forceinline__ void for_runs(const Segments &g, int b0, int b1, F &&f) {
    const int lane = threadIdx.x & 63;
    int at = b0;
    auto run = [&](int start, int end, int id) __attribute__((always_inline)) {
        const int lo = min(max(start, at), b1), hi = min(max(end, lo), b1);
        if (lo > at) f(-1, at, lo);
        if (hi > lo) f(id >= 0 && id < g.adapters ? id : -1, lo, hi);
        at = hi;
    };
    int s = 0, n = g.count;
    if (n <= 64) {
        // a lane a segment: one access to memory before the first run
        const bool mine = lane < n;
        const int start = mine ? g.offsets[lane] : 0, end = mine ? g.offsets[lane + 1] : 0, id = mine ? g.ids[lane] : -1;
        for (uint64_t rest = __ballot(mine && end > b0 && start < b1); rest && at < b1; rest &= rest - 1) {
            const int k = __builtin_ctzll(rest);
            run(__builtin_amdgcn_readlane(start, k), __builtin_amdgcn_readlane(end, k), __builtin_amdgcn_readlane(id, k));
        }
    } else {
        // the first segment that ends past b0, by a search over 64 parts at a time
        while (n > 0) {
            const int step = (n + 63) / 64, probe = (lane + 1) * step - 1;
            const bool before = probe < n && g.offsets[s + probe + 1] <= b0;
            const int parts = __builtin_popcountll(__ballot(before));
            s += parts * step;
            n = min(step - 1, n - parts * step);
        }
        for (; at < b1 && s < g.count; ++s) run(g.offsets[s], g.offsets[s + 1], g.ids[s]);
    }
    if (at < b1) f(-1, at, b1);
}

// ---- shrink --------------------------------------------------------------------------------

struct ShrinkArgs {
    const uint16_t *X, *A;  // rows [T][ldx], adapters [N][r][K]
    int64_t ldx;
    const float *scales;  // null: one
    float *U;             // [parts][r][T]
    Segments seg;
    int32_t K, r, block, parts;  // rows a workgroup; shares of the reduction
};

__device__ __forceinline__ void zero_u(float *U, int r, int ld, int lo, int hi) {
    const int rows = hi - lo;
    for (int i = threadIdx.x; i < r * rows; i += 256) U[(int64_t)(i / rows) * ld + lo + i % rows] = 0.f;
}

// For a few rows each: `block` rows (at most 16) by 16 QF ranks at a time a workgroup,
// one part of the reduction, which its four waves share.  (64 rows of 64 adapters, 8192
// columns, r = 16, eight parts: 6.1 us, bound by the launch and one latency of memory.)
template <typename T, int QF>
__global__ __launch_bounds__(256) void shrink_kernel(ShrinkArgs a) {
    constexpr int PF = 1;
    __shared__ f32x4 sums[4][QF][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int b0 = blockIdx.x * a.block, b1 = min(b0 + a.block, a.seg.rows);
    const int steps = (a.K + 31) / 32;
    const int from = (int)((int64_t)steps * blockIdx.y / a.parts), to = (int)((int64_t)steps * (blockIdx.y + 1) / a.parts);
    const int share = (to - from + 3) / 4, s0 = from + wave * share, s1 = min(s0 + share, to);
    float *U = a.U + (int64_t)blockIdx.y * a.r * a.seg.rows;
    for_runs(a.seg, b0, b1, [&](int n, int lo, int hi) __attribute__((always_inline)) {
        if (n < 0) return zero_u(U, a.r, a.seg.rows, lo, hi);
        const float scale = a.scales ? a.scales[n] : 1.f;
        uint32_t xo[PF];
        fragment_offsets(hi - lo, a.ldx, xo);
        for (int r0 = 0; r0 < a.r; r0 += 16 * QF) {
            uint32_t ao[QF];
            fragment_offsets(a.r - r0, a.K, ao);
            f32x4 acc[QF][PF] = {};
            stream_product<T, QF, PF, 4>(buffer_of(a.A + ((int64_t)n * a.r + r0) * a.K), ao,
                                                             buffer_of(a.X + lo * a.ldx), xo, s0, s1, a.K, acc);
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
                const int rank = r0 + 16 * (f / PF) + 4 * (ln >> 4), row = lo + 16 * (f % PF) + (ln & 15);
                if (row < hi) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (rank + e < a.r) U[(int64_t)(rank + e) * a.seg.rows + row] = v[e] * scale;
                }
            }
            __syncthreads();
        }
    });
}

// For many rows: 64 a workgroup, 16 a wave, by 16 QF ranks at a time.  X and A_n are
// copied into LDS in steps of 64 reduction values (whole lines of 128 bytes, as
// RcOperand's), DEPTH steps at a time; a wave copies its own rows of X and a quarter of
// A_n's.  (Reading fragments of 16 rows by 64 bytes straight into registers, 32768 rows
// of 8192 took 148 us with r = 32, 20011 rows 95 with r = 16.)
template <typename T, int QF>
__global__ __launch_bounds__(256) void shrink_block_kernel(ShrinkArgs a) {
    constexpr int DEPTH = QF == 1 ? 6 : QF == 2 ? 5 : 4;
    constexpr int XB = 64 * 128, AB = 16 * QF * 128, STAGE = XB + AB;
    constexpr int NA = QF <= 2 ? 1 : QF / 2;  // copies of A_n a wave and step (half a copy with QF = 1)
    constexpr int NC = 2 + NA;
    __shared__ __attribute__((aligned(1024))) char lds[DEPTH * STAGE];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int b0 = blockIdx.x * a.block, b1 = min(b0 + a.block, a.seg.rows);
    const int all = (a.K + 63) / 64;
    const int from = (int)((int64_t)all * blockIdx.y / a.parts), steps = (int)((int64_t)all * (blockIdx.y + 1) / a.parts) - from;
    float *U = a.U + (int64_t)blockIdx.y * a.r * a.seg.rows;
    const uint32_t at = lds_addr(lds);
    // Each workgroup begins at another step: where rows are a power of two apart, the
    // same columns of all rows lie in few of the memory's channels.
    const int turn = (int)((int64_t)steps * blockIdx.x / gridDim.x);
    // a copy is 8 rows of 128 bytes: lane l has chunk (l % 8) ^ (row / 2 % 8) of row l / 8
    const int row8 = lane >> 3, a_first = QF == 1 ? wave * 4 : wave * 8 * NA;
    uint32_t xf[2], af[2];  // this lane's fragments of the two halves of a step, within a stage
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int slot = (4 * h + g) ^ ((c >> 1) & 7);
        xf[h] = (uint32_t)((16 * wave + c) * 128 + slot * 16);
        af[h] = (uint32_t)(XB + c * 128 + slot * 16);
    }
    for_runs(a.seg, b0, b1, [&](int n, int lo, int hi) __attribute__((always_inline)) {
        if (n < 0) return zero_u(U, a.r, a.seg.rows, lo, hi);
        const float scale = a.scales ? a.scales[n] : 1.f;
        const int mine = lo + 16 * wave;  // this wave's rows
        for (int r0 = 0; r0 < a.r; r0 += 16 * QF) {
            uint32_t xo[2], ao[NA], xk[2], ak[NA];  // offsets of a lane's copies, and their first reduction values
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int row = 8 * j + row8;
                xk[j] = (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) * 8);
                xo[j] = mine + row < hi ? (uint32_t)((row * a.ldx + xk[j]) * 2) : kOOB;
            }
#pragma unroll
            for (int j = 0; j < NA; ++j) {
                const int row = a_first + 8 * j + row8;
                ak[j] = (uint32_t)(((lane & 7) ^ ((row >> 1) & 7)) * 8);
                ao[j] = r0 + row < a.r ? (uint32_t)(((int64_t)row * a.K + ak[j]) * 2) : kOOB;
            }
            const rsrc_t xr = make_rsrc(reinterpret_cast<const char *>(a.X + (mine < hi ? mine : lo) * a.ldx));
            const rsrc_t ar = make_rsrc(reinterpret_cast<const char *>(a.A + ((int64_t)n * a.r + r0) * a.K));
            auto issue = [&](int s) __attribute__((always_inline)) {  // past the last step: zeros
                const uint32_t stage = at + (uint32_t)(s % DEPTH) * STAGE;
                const int turned = s + turn < steps ? s + turn : s + turn - steps;
                const uint32_t k0 = s < steps ? (uint32_t)(from + turned) * 64 : (uint32_t)a.K;
                const uint32_t left = (uint32_t)a.K - k0;
#pragma unroll
                for (int j = 0; j < 2; ++j) copy16(xr, stage + wave * 2048 + j * 1024, xk[j] < left ? xo[j] + k0 * 2 : kOOB);
                if constexpr (QF == 1) {
                    if (lane < 32) copy16(ar, stage + XB + wave * 512, ak[0] < left ? ao[0] + k0 * 2 : kOOB);
                } else {
#pragma unroll
                    for (int j = 0; j < NA; ++j)
                        copy16(ar, stage + XB + (wave * NA + j) * 1024, ak[j] < left ? ao[j] + k0 * 2 : kOOB);
                }
            };
            f32x4 acc[QF] = {};
#pragma unroll
            for (int s = 0; s < DEPTH - 1; ++s) issue(s);
            for (int s = 0; s < steps; ++s) {
                // step s has landed, and every wave has read step s - 1
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((DEPTH - 2) * NC) : "memory");
                issue(s + DEPTH - 1);
                const uint32_t stage = at + (uint32_t)(s % DEPTH) * STAGE;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const u32x4 x = *reinterpret_cast<const __attribute__((address_space(3))) u32x4 *>((uintptr_t)(stage + xf[h]));
#pragma unroll
                    for (int i = 0; i < QF; ++i)
                        acc[i] = mfma<T>(
                            *reinterpret_cast<const __attribute__((address_space(3))) u32x4 *>((uintptr_t)(stage + af[h] + i * 2048)), x,
                            acc[i]);
                }
            }
            // every copy has landed and every read returned, before LDS is filled again
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
            for (int i = 0; i < QF; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int rank = r0 + 16 * i + 4 * g + e, row = mine + c;
                    if (rank < a.r && row < hi) U[(int64_t)rank * a.seg.rows + row] = acc[i][e] * scale;
                }
        }
    });
}

// ---- expand --------------------------------------------------------------------------------

struct ExpandArgs {
    const float *U;       // [parts][r][T]; parts and U_out: of expand_row_kernel
    float *U_out;         // the parts' sum, or null
    const uint16_t *B;    // [N][r][M]
    const float *scales;  // null: one
    const void *Y0;       // null: zero
    void *Y;
    int64_t ldy0, ldy;
    Segments seg;
    int32_t M, r, parts;
    int32_t same;  // Y is Y0: rows without an adapter are left
};

template <typename YT>
__device__ __forceinline__ void load_y(const ExpandArgs &a, int64_t row, int64_t m, float (&v)[8]) {
    if (a.Y0) {
        load8(static_cast<const YT *>(a.Y0) + row * a.ldy0 + m, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
}

// U[rank][row] as the sum of its parts, in order.
__device__ __forceinline__ float u_at(const ExpandArgs &a, int rank, int row) {
    const float *p = a.U + (int64_t)rank * a.seg.rows + row;
    float u = 0.f;
    for (int k0 = 0; k0 < a.parts; k0 += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = k0 + k < a.parts ? p[(int64_t)(k0 + k) * a.r * a.seg.rows] : 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) u += v[k];
    }
    return u;
}

typedef int16_t s16x8 __attribute__((ext_vector_type(8)));
template <typename T>
constexpr int16_t kInf16 = std::is_same<T, f16_t>::value ? 0x7c00 : 0x7f80;

// Eight fp32 values in planes of the 16-bit type that the other operand has, so that the
// 16-bit instruction multiplies them: three of bf16 (24 bits, at any scale), two of fp16
// under a scale 2^(15 - e) that takes the largest of those that share it into [2^14, 2^15).
// The second fp16 plane's unit is 2^-24: half of it is 2^-39 of the largest, and down to
// 2^-17 of the largest it is no more than the second rounding, 2^-22 of the value.
template <typename T>
struct Planes;
template <>
struct Planes<bf16_t> {
    static constexpr int N = 3;
    static constexpr bool kScaled = false;
};
template <>
struct Planes<f16_t> {
    static constexpr int N = 2;
    static constexpr bool kScaled = true;
};
// An infinity among the other operand's elements makes the sum of the planes' products NaN
// where it should be the infinity: the planes past the first may be zero, or of the other
// sign.  So sums that are not finite are formed once more (expand in fp32, grad as below);
// what a finite product takes does not change.
//
// ODD: for products with infinities.  The first plane of a value x (v is x scaled) is neither
// zero nor an infinity where x is not (fp32's largest values round up past bf16's), and the
// others are given finite_only of the other operand, zeros in place of its infinities and
// NaN.  (Always so, the gradient of 16384 fp16 rows of 4096, r = 48, took 318 us in place of
// 260.)
template <bool ODD, typename T, int N>
__device__ __forceinline__ void split_planes(const float (&x)[8], const float (&v)[8], u32x4 (&out)[N]) {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
    for (int p = 0; p < N; ++p) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            uint32_t b[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                b[q] = bits16<T>(r[2 * h + q]);
                if (ODD && p == 0) {
                    const uint32_t least = min(__builtin_bit_cast(uint32_t, x[2 * h + q]) << 1, 1u);
                    uint32_t size = max(b[q] & 0x7fffu, least);
                    if (!Planes<T>::kScaled && size == (uint32_t)kInf16<T>)  // cut off, not rounded
                        size = __builtin_bit_cast(uint32_t, r[2 * h + q]) >> 16 & 0x7fffu;
                    b[q] = (b[q] & 0x8000u) | size;
                }
                const float rest = r[2 * h + q] - value16<T>(b[q]);
                r[2 * h + q] = fabsf(rest) < INFINITY ? rest : 0.f;  // nothing is left of an infinity or a NaN
            }
            out[p][h] = b[0] | (b[1] << 16);
        }
    }
}

template <typename T>
__device__ __forceinline__ u32x4 finite_only(u32x4 x) {
    const s16x8 v = __builtin_bit_cast(s16x8, x);
    const s16x8 keep = ((v & (int16_t)0x7fff) - kInf16<T>) >> (int16_t)15;
    return __builtin_bit_cast(u32x4, v & keep);
}

// A value's part in the largest of those that share a scale: an infinity (or NaN) has
// none, so that it takes no finite value past the type's range.
__device__ __forceinline__ float largest_of(float most, float x) {
    return fabsf(x) < INFINITY ? fmaxf(most, fabsf(x)) : most;
}
// The exponent e of that scale for the largest of `most` over the wave's lanes of equal
// lane % 16 (not so low that 2^(e - 15) is no normal number).
__device__ __forceinline__ int scale_exponent(float most) {
    most = fmaxf(most, __shfl_xor(most, 16, 64));
    most = fmaxf(most, __shfl_xor(most, 32, 64));
    return max(__builtin_amdgcn_frexp_expf(most), -110);
}

// Whether any lane has a sum that is infinite or NaN.
template <int N>
__device__ __forceinline__ bool any_infinite(const f32x4 (&acc)[N]) {
    float none[8] = {};  // eight chains
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) none[4 * (j & 1) + e] = __builtin_fmaf(acc[j][e], 0.f, none[4 * (j & 1) + e]);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += none[i];
    return __ballot(sum != 0.f) != 0;  // NaN
}

// A wave: 128 columns of a run of rows, 16 rows at a time.  Per step of 32 ranks a lane
// reads eight columns of eight rows of B_n and turns them, in its own registers, into one
// operand for each of the columns, held over the run (STEPS of 1 or 2, r <= 64; with 0,
// more ranks, read again for every 16 rows); of U it has eight ranks of a row, split into
// planes.  Instruction j gives rows 4 (lane / 16) .. +3 of column 8 (lane % 16) + j, so
// that a lane has eight consecutive columns of Y.  U and Y0 of the next 16 rows are on
// their way while these are multiplied and stored.  (On the fp32 instruction, 4508 rows
// of 2384 in 61 segments, r = 64, took 50 us, 37 so; 32768 of 8192 into fp32, r = 32, 462
// and 406.)
// With one step held two waves a SIMD fit: their bound keeps the sums' second form, which is
// hardly ever run, from costing registers.
constexpr int kExpandCols = 512;
template <typename T, typename YT, int STEPS>
__global__ __launch_bounds__(256, STEPS == 1 ? 2 : 1) void expand_kernel(ExpandArgs a, int block) {
    constexpr int NP = Planes<T>::N, HELD = STEPS > 0 ? STEPS : 1;
    constexpr bool kScaled = Planes<T>::kScaled;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 15, g = lane >> 4;
    const int b0 = blockIdx.x * block, b1 = min(b0 + block, a.seg.rows);
    const int m = blockIdx.y * kExpandCols + wave * 128 + 8 * c;
    const bool in = m < a.M;
    for_runs(a.seg, b0, b1, [&](int n, int lo, int hi) __attribute__((always_inline)) {
        if (n < 0) {
            if (a.same || !in) return;
            for (int row = lo + g; row < hi; row += 4) {
                float y[8];
                load_y<YT>(a, row, m, y);
                store8(static_cast<YT *>(a.Y) + row * a.ldy + m, y);
            }
            return;
        }
        const float scale = a.scales ? a.scales[n] : 1.f;
        const uint16_t *B = a.B + (int64_t)n * a.r * a.M + m;
        u32x4 b[HELD][8];  // column j's eight ranks of each step
        auto load_b = [&](int s, int r0) __attribute__((always_inline)) {
            u32x4 raw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int rank = r0 + 8 * g + i;
                raw[i] = u32x4{0, 0, 0, 0};
                if (in && rank < a.r) raw[i] = *reinterpret_cast<const u32x4 *>(B + (int64_t)rank * a.M);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int h = 0; h < 4; ++h)  // the low or the high halves of two rows' words
                    b[s][j][h] = __builtin_amdgcn_perm(raw[2 * h + 1][j >> 1], raw[2 * h][j >> 1], j & 1 ? 0x07060302u : 0x05040100u);
        };
        auto load_u = [&](int row0, int r0, float (&u)[8]) __attribute__((always_inline)) {
            const int row = row0 + c;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int rank = r0 + 8 * g + i;
                u[i] = row < hi && rank < a.r ? a.U[(int64_t)rank * a.seg.rows + row] : 0.f;
            }
        };
        auto load_y0 = [&](int row0, Raw8<YT> (&out)[4]) __attribute__((always_inline)) {
            if (!a.Y0 || !in) return;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                out[e].load(static_cast<const YT *>(a.Y0) + min(row0 + 4 * g + e, hi - 1) * a.ldy0 + m);
        };
        // acc += the product of 32 ranks of U, whose rows have the exponent e
        auto multiply = [&](float (&u)[8], int s, int e, f32x4 (&acc)[8]) __attribute__((always_inline)) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = kScaled ? ldexpf(u[i] * scale, 15 - e) : u[i] * scale;
            u32x4 pl[NP];
            split_planes<false, T>(v, v, pl);
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int p = 0; p < NP; ++p) acc[j] = mfma<T>(pl[p], b[s][j], acc[j]);
        };
        // Where a sum is infinite or NaN, the same in fp32, a rank after another: planes do not
        // multiply infinities.  (Under a scale no finite product comes near fp32's range, so that
        // this sum is not finite either, and the scale changes nothing.)
        auto in_f32 = [&](int row0, f32x4 (&acc)[8]) __attribute__((always_inline)) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = row0 + 4 * g + q;
                float d[8] = {};
#pragma unroll 1
                for (int k = 0; k < (in && row < hi ? a.r : 0); ++k) {
                    float x[8];
                    load8(reinterpret_cast<const T *>(B + (int64_t)k * a.M), x);
                    const float w = a.U[(int64_t)k * a.seg.rows + row] * scale;
#pragma unroll
                    for (int e = 0; e < 8; ++e) d[e] += w * x[e];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j][q] = fabsf(acc[j][q]) < INFINITY ? acc[j][q] : d[j];
            }
        };
        auto largest = [&](float (&u)[8], float most) __attribute__((always_inline)) -> float {
#pragma unroll
            for (int i = 0; i < 8; ++i) most = largest_of(most, u[i] * scale);
            return most;
        };
        auto rows16 = [&](int row0, float (&u)[HELD][8], Raw8<YT> (&y0)[4]) __attribute__((always_inline)) {
            f32x4 acc[8] = {};
            int e = 0;
            if constexpr (kScaled) {
                float most = 0.f;
                if constexpr (STEPS > 0) {
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) most = largest(u[s], most);
                } else {
                    for (int r0 = 0; r0 < a.r; r0 += 32) {
                        load_u(row0, r0, u[0]);
                        most = largest(u[0], most);
                    }
                }
                e = scale_exponent(most);
            }
            if constexpr (STEPS > 0) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s) multiply(u[s], s, e, acc);
            } else {
                for (int r0 = 0; r0 < a.r; r0 += 32) {
                    load_b(0, r0);
                    load_u(row0, r0, u[0]);
                    multiply(u[0], 0, e, acc);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            asm volatile("s_nop 7" ::: "memory");  // the last products, before anything reads the sums
            if (__builtin_expect(any_infinite(acc), 0)) in_f32(row0, acc);
            const float back = kScaled ? ldexpf(1.f, e - 15) : 1.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = row0 + 4 * g + q;
                const float f = kScaled ? __shfl(back, 4 * g + q, 64) : 1.f;
                float o[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = acc[j][q] * f + (a.Y0 ? y0[q][j] : 0.f);
                if (in && row < hi) stream8(static_cast<YT *>(a.Y) + row * a.ldy + m, o);
            }
        };
        Raw8<YT> y[2][4];
        float u[2][HELD][8];
        auto fetch = [&](int row0, float (&to)[HELD][8], Raw8<YT> (&y0)[4]) __attribute__((always_inline)) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) load_u(row0, 32 * s, to[s]);
            load_y0(row0, y0);
        };
#pragma unroll
        for (int s = 0; s < STEPS; ++s) load_b(s, 32 * s);
        fetch(lo, u[0], y[0]);
        for (int row = lo; row < hi; row += 32) {
            fetch(row + 16, u[1], y[1]);
            rows16(row, u[0], y[0]);
            if (row + 16 >= hi) break;
            fetch(row + 32, u[0], y[0]);
            rows16(row + 16, u[1], y[1]);
        }
    });
}

// One row by 2048 columns, for segments of a token or so: the multiplications are few,
// and B_n is read once, eight columns a thread, sixteen ranks in flight.  (64 rows of 64
// adapters, 8192 columns, r = 16: 5.8 us, bound by the launch and one latency of memory.)
constexpr int kMostRank = 256;
template <typename T, typename YT>
__global__ __launch_bounds__(256) void expand_row_kernel(ExpandArgs a) {
    __shared__ float u[kMostRank];
    const int row = blockIdx.x;
    const int m = (blockIdx.y * 256 + threadIdx.x) * 8;
    for_runs(a.seg, row, row + 1, [&](int n, int lo, int hi) __attribute__((always_inline)) {
        (void)lo;
        (void)hi;
        if (n < 0 && a.same && !a.U_out) return;
        const bool in = m < a.M;
        const T *B = reinterpret_cast<const T *>(a.B + (int64_t)(n < 0 ? 0 : n) * a.r * a.M + (in ? m : 0));
        float y[8], d[8] = {};
        u32x4 raw[16];
        auto load_b = [&](int k) __attribute__((always_inline)) {
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                raw[q] = u32x4{0, 0, 0, 0};
                if (k + q < a.r) raw[q] = *reinterpret_cast<const u32x4 *>(B + (int64_t)(k + q) * a.M);
            }
        };
        // what the row needs of B_n and Y0 is on its way before U is read
        if (n >= 0) load_b(0);
        if (in) load_y<YT>(a, row, m, y);
        const float scale = n >= 0 && a.scales ? a.scales[n] : 1.f;
        for (int i = threadIdx.x; i < a.r; i += 256) {
            const float v = n >= 0 ? u_at(a, i, row) : 0.f;
            if (a.U_out && blockIdx.y == 0) a.U_out[(int64_t)i * a.seg.rows + row] = v;
            u[i] = v * scale;
        }
        __syncthreads();
        if (!in || (n < 0 && a.same)) return;
        for (int k = 0; n >= 0 && k < a.r; k += 16) {
            if (k > 0) load_b(k);
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                if (k + q >= a.r) break;
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] += u[k + q] * value16<T>((raw[q][e >> 1] >> (16 * (e & 1))) & 0xffffu);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] += d[e];
        store8(static_cast<YT *>(a.Y) + row * a.ldy + m, y);
    });
}

// ---- grad ----------------------------------------------------------------------------------

// One of the two gradients that a launch forms.
struct GradOf {
    const float *V;     // [r][T]
    const uint16_t *X;  // [T][ldx]
    int64_t ldx;
    const float *scales;  // null: one
    float *G;             // [N][r][K]
    float *part;          // the first split's sums, [N][r][K], where there are several
    int32_t K;
};
struct GradArgs {
    GradOf of[2];
    int64_t part_split;  // from one split's sums to the next one's
    Segments seg;
    int32_t tiles0;      // column tiles of of[0]
    int32_t r, splits, accumulate;
};

// One adapter by 128 columns of one of the two gradients by 16 F ranks a workgroup, over
// one split of the adapter's rows (columns first in the grid, so that every XCD gets its
// share of each adapter).
// Its four waves take chunks of 32 rows in turn, each by itself: the chunk's columns are
// copied into the wave's part of LDS (16 bytes a lane, whole rows of 256 bytes), the
// next chunk's while this one is multiplied, and read back across the rows
// (ds_read_b64_tr_b16); V comes to registers as eight rows of a rank a lane.  (32768 rows
// of 8192 and 8192 with r = 32: 237 us, 4.5 TB/s; in two launches with two splits 138 each,
// and 6 for their sum.  In fp32, 16 x 16 x 4 at a time, each took 183, 109 of them the
// matrix cores' at their rate.)  A wave whose sums are not finite forms them again, as ODD
// products.  (Two waves a SIMD fit, but for four fragments of fp16.)
template <typename T, int F>
__global__ __launch_bounds__(256, Planes<T>::kScaled ? 1 : 2) void grad_kernel(GradArgs a) {
    constexpr int NP = Planes<T>::N;
    constexpr bool kScaled = Planes<T>::kScaled;
    constexpr int kChunk = 32, kRowB = 256, kStage = kChunk * kRowB;
    __shared__ __attribute__((aligned(1024))) char lds[4 * 2 * kStage];
    __shared__ int any[4];  // of each wave: it has multiplied rows
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;
    const int n = blockIdx.y / a.splits, split = blockIdx.y % a.splits;
    const bool second = (int)blockIdx.x >= a.tiles0;
    const GradOf &d = a.of[second];
    const int64_t ldx = d.ldx;
    const int K = d.K, k0 = ((int)blockIdx.x - (second ? a.tiles0 : 0)) * 128, r0 = blockIdx.z * (16 * F);
    const uint16_t *X = d.X + k0;
    char *mine = lds + wave * (2 * kStage);
    const uint32_t at = lds_addr(mine);

    // Copy i of a chunk fills its rows 4 i .. 4 i + 3, 16 lanes a row.  The 32-byte
    // segments of a row are permuted as in RsOperand, so that a transposing read falls
    // on distinct banks.
    auto swizzle = [](int row) { return (row & 3) | ((row >> 1) & 4); };
    uint32_t xo[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 4 * i + g, col = ((((c >> 1) ^ swizzle(row)) << 1) | (c & 1)) * 8;
        xo[i] = k0 + col < K ? (uint32_t)((row * ldx + col) * 2) : kOOB;
    }
    // fragment 0 (16 columns): this lane's part of rows 0 .. 3 of each eight; the others are 4
    // rows on, and fragment j's at the address with bits 5 .. 7 changed by j
    const int kl = 8 * g + (c >> 2);
    const uint32_t fo = (uint32_t)(kl * kRowB + (swizzle(kl) << 5) + 8 * (c & 3));
    // ranks past the last read the last one's values and are not stored
    const float *V[F];
#pragma unroll
    for (int f = 0; f < F; ++f) V[f] = d.V + (int64_t)min(r0 + 16 * f + c, a.r - 1) * a.seg.rows;

    // The chunks of this wave: the workers (waves of all splits) take the adapter's chunks
    // in turn, across its segments, so that short ones are shared out too (4508 rows in
    // 61 segments of 3 adapters, r = 64: 204 us for the whole gradient when each segment
    // began with the first worker).  `due`: chunks of the next segment before this
    // wave's first.
    const int workers = 4 * a.splits, step = workers * kChunk;
    int s0, hi, t, due;
    uint64_t left;
    auto next = [&]() __attribute__((always_inline)) -> bool {
        t += step;
        while (t >= hi) {
            while (!left) {
                s0 += 64;
                if (s0 >= a.seg.count) return false;
                left = __ballot(s0 + lane < a.seg.count && a.seg.ids[min(s0 + lane, a.seg.count - 1)] == n);
            }
            const int s = s0 + __builtin_ctzll(left);
            left &= left - 1;
            const int lo = min(max(a.seg.offsets[s], 0), a.seg.rows);
            hi = min(max(a.seg.offsets[s + 1], lo), a.seg.rows);
            t = lo + due * kChunk;
            due -= (hi - lo + kChunk - 1) / kChunk % workers;
            due += due < 0 ? workers : 0;
        }
        return true;
    };
    auto copy = [&](int stage) __attribute__((always_inline)) {
        const rsrc_t rs = make_rsrc(reinterpret_cast<const char *>(X + t * ldx));
        if (t + kChunk <= hi) {
#pragma unroll
            for (int i = 0; i < 8; ++i) copy16(rs, at + stage * kStage + i * 1024, xo[i]);
        } else {  // rows past the segment read as zero
#pragma unroll
            for (int i = 0; i < 8; ++i) copy16(rs, at + stage * kStage + i * 1024, t + 4 * i + g < hi ? xo[i] : kOOB);
        }
    };
    float v[F][8];
    auto load_v = [&]() __attribute__((always_inline)) {
        const int row = t + 8 * g;
        if (t + kChunk <= hi) {
#pragma unroll
            for (int f = 0; f < F; ++f) load8(V[f] + row, v[f]);
        } else {
#pragma unroll
            for (int f = 0; f < F; ++f)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[f][i] = row + i < hi ? V[f][row + i] : 0.f;
        }
    };

    f32x4 acc[F][8];
    auto sum = [&](auto odd) __attribute__((always_inline)) {
        constexpr bool ODD = decltype(odd)::value;
        s0 = -64, hi = 0, t = -step, due = split * 4 + wave;
        left = 0;
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        int stage = 0;
        bool more = next();
        if (lane == 0) any[wave] = more;
        if (more) {
            copy(0);
            load_v();
        }
        while (more) {
            // this chunk is in LDS, its V in registers, and the other stage has been read
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
            u32x4 pl[F][NP];
            [[maybe_unused]] float unscale[F][4];
#pragma unroll
            for (int f = 0; f < F; ++f) {
                float w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = v[f][i];
                if constexpr (kScaled) {
                    float most = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) most = largest_of(most, w[i]);
                    const int e = scale_exponent(most);  // of the rank's 32 rows
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = ldexpf(w[i], 15 - e);
                    const float back = ldexpf(1.f, e - 15);
#pragma unroll
                    for (int i = 0; i < 4; ++i) unscale[f][i] = __shfl(back, 4 * g + i, 64);
                }
                split_planes<ODD, T>(v[f], w, pl[f]);
            }
            more = next();
            if (more) {
                copy(stage ^ 1);
                load_v();
            }
            const uint32_t base = at + stage * kStage + fo;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t from = base ^ (uint32_t)(j << 5);
                const s16x4 x0 =
                    __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(uintptr_t)from);
                const s16x4 x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4 *)(uintptr_t)(from + 4 * kRowB));
                const u32x2 w0 = __builtin_bit_cast(u32x2, x0), w1 = __builtin_bit_cast(u32x2, x1);
                const u32x4 x = {w0[0], w0[1], w1[0], w1[1]}, rest = ODD ? finite_only<T>(x) : x;
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    if constexpr (kScaled) {
                        f32x4 part = {};
#pragma unroll
                        for (int p = 0; p < NP; ++p) part = mfma<_Float16>(pl[f][p], p ? rest : x, part);
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[f][j][e] += part[e] * unscale[f][e];
                    } else {
#pragma unroll
                        for (int p = 0; p < NP; ++p) acc[f][j] = mfma<__bf16>(pl[f][p], p ? rest : x, acc[f][j]);
                    }
                }
            }
            stage ^= 1;
        }
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_nop 7\n\ts_nop 7" ::: "memory");  // the last products, before anything reads the sums
    };
    sum(std::integral_constant<bool, false>{});
    bool infinite = false;
#pragma unroll
    for (int f = 0; f < F; ++f) infinite |= any_infinite(acc[f]);
    if (__builtin_expect(infinite, 0)) sum(std::integral_constant<bool, true>{});

    // the four waves' sums meet in LDS, one fragment of ranks at a time
    const float scale = d.scales ? d.scales[n] : 1.f;
    const bool whole = a.splits == 1, adds = whole && a.accumulate;
    // Without rows nothing is scaled, whatever the scale; -0 added to what was there
    // leaves its bits.
    const float none = a.accumulate ? -0.f : 0.f;
    float *out = (whole ? d.G : d.part + split * a.part_split) + (int64_t)n * a.r * K;
    f32x4(*sums)[8][64] = reinterpret_cast<f32x4(*)[8][64]>(lds);
#pragma unroll
    for (int f = 0; f < F; ++f) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[wave][j][lane] = acc[f][j];
        __syncthreads();
        const bool rows = any[0] | any[1] | any[2] | any[3];
        // thread (lane, wave): rank 4 (lane / 16) + wave of the fragment, columns 16 j + lane % 16
        const int rank = r0 + 16 * f + 4 * g + wave;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float sum = sums[0][j][lane][wave];
#pragma unroll
            for (int k = 1; k < 4; ++k) sum += sums[k][j][lane][wave];
            const int col = k0 + 16 * j + c;
            if (col < K && rank < a.r) {
                float *p = out + (int64_t)rank * K + col;
                if (rows) *p = (adds ? *p : 0.f) + sum * scale;
                else if (!adds) *p = none;
            }
        }
    }
}

// out[i] (+)= the sum of part[p stride + i] over the parts p, in order, for two arrays,
// one behind the other in each part: n values of out, n2 of out2 (0: none).
__global__ __launch_bounds__(256) void sum_parts_kernel(const float *part, int parts, int64_t stride, int64_t n, float *out, int64_t n2,
                                                        float *out2, int accumulate) {
    const int64_t groups = (n + 7) / 8;
    int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const bool second = i >= groups;
    if (second) {
        i -= groups;
        part += n;
        out = out2;
    }
    i *= 8;
    const int64_t left = (second ? n2 : n) - i;
    if (left <= 0) return;
    float sum[8], v[8];
    load_n(part + i, left, sum);
    for (int p = 1; p < parts; ++p) {
        load_n(part + p * stride + i, left, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += v[e];
    }
    if (accumulate) {
        load_n(out + i, left, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = v[e] + sum[e];
    }
    store_n(out + i, left, sum);
}

// ---- launches ------------------------------------------------------------------------------

// Rows a workgroup of shrink: one where segments are of a token or so.
int block_of(int64_t T, int64_t S) {
    const int64_t mean = T / S;
    return mean < 4 ? 1 : mean <= 32 ? 16 : 64;
}
// Shares of the reduction, so that a few rows still occupy the chip, and a block that
// takes two passes, where segments meet, holds up little: at least 512 columns each.
// (20011 rows of 8192 in 29 segments, 313 blocks: 101 us in one share, 76 in three.)
constexpr int64_t kMostParts = 16;
int64_t parts_of(int64_t T, int64_t S, int64_t K) {
    const int64_t block = block_of(T, S), groups = block == 1 ? 512 : 1024;
    return max64(1, min64(min64(groups / ceil_div(T, block), kMostParts), K / 512));
}
// The shares' sums for T or any fewer rows (of blocks of at most 64).
uint64_t parts_bytes(int64_t T, int64_t r) { return round_up((uint64_t)max64(T, min64(kMostParts * T, 64 * 1024)) * (uint64_t)r * 4); }
uint64_t u_bytes(int64_t T, int64_t r) { return round_up((uint64_t)T * (uint64_t)r * 4); }

// Splits of the adapters' rows, so that a few adapters still occupy the chip (two
// workgroups a compute unit), each of a thousand rows or more.
constexpr int64_t kGradGroups = 512;
int64_t splits_of(int64_t T, int64_t N, int64_t tiles) { return max64(1, min64(kGradGroups / (N * tiles), ceil_div(T, 1024))); }
uint64_t part_bytes(int64_t r) { return (uint64_t)kGradGroups * 128 * (uint64_t)r * 4; }

template <typename T, int QF>
hipError_t shrink_blocks(const ShrinkArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)ceil_div(a.seg.rows, a.block), (unsigned)a.parts);
    if (a.block <= 16)
        hipLaunchKernelGGL((shrink_kernel<T, QF>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((shrink_block_kernel<T, QF>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}
hipError_t shrink(int dtype, const ShrinkArgs &a, hipStream_t s) {
    auto go = [&](auto type) {
        using T = decltype(type);
        return a.r <= 16 ? shrink_blocks<T, 1>(a, s) : a.r <= 32 ? shrink_blocks<T, 2>(a, s) : shrink_blocks<T, 4>(a, s);
    };
    return dtype == ZI_F16 ? go(f16_t{}) : go(bf16_t{});
}

constexpr int64_t kExpandGroups = 512;
template <typename T, typename YT>
hipError_t expand_typed(const ExpandArgs &a, bool rows, hipStream_t s) {
    if (rows)
        hipLaunchKernelGGL((expand_row_kernel<T, YT>), dim3((unsigned)a.seg.rows, (unsigned)ceil_div(a.M, 2048)), dim3(256), 0, s, a);
    else {
        const int64_t wide = ceil_div(a.M, kExpandCols);
        int block = 128;  // rows a workgroup: fewer where the chip would not be full
        while (block > 16 && ceil_div(a.seg.rows, block) * wide < kExpandGroups) block /= 2;
        const dim3 grid((unsigned)ceil_div(a.seg.rows, block), (unsigned)wide);
        auto go = [&](auto hold) {
            hipLaunchKernelGGL((expand_kernel<T, YT, decltype(hold)::value>), grid, dim3(256), 0, s, a, block);
        };
        if (a.r <= 32) go(std::integral_constant<int, 1>{});
        else if (a.r <= 64) go(std::integral_constant<int, 2>{});
        else go(std::integral_constant<int, 0>{});
    }
    return hipGetLastError();
}
hipError_t expand(int dtype, int out_dtype, const ExpandArgs &a, bool rows, hipStream_t s) {
    if (dtype == ZI_F16) return out_dtype == ZI_F32 ? expand_typed<f16_t, float>(a, rows, s) : expand_typed<f16_t, f16_t>(a, rows, s);
    return out_dtype == ZI_F32 ? expand_typed<bf16_t, float>(a, rows, s) : expand_typed<bf16_t, bf16_t>(a, rows, s);
}

hipError_t sum_parts(const float *part, int64_t parts, int64_t n, float *out, int64_t n2, float *out2, int accumulate, hipStream_t s) {
    hipLaunchKernelGGL(sum_parts_kernel, dim3((unsigned)ceil_div(ceil_div(n, 8) + ceil_div(n2, 8), 256)), dim3(256), 0, s, part,
                       (int)parts, n + n2, n, out, n2, out2, accumulate);
    return hipGetLastError();
}

hipError_t grad(int dtype, const GradArgs &a, int64_t tiles, hipStream_t s) {
    auto go = [&](auto type, auto frags) {
        constexpr int F = decltype(frags)::value;
        hipLaunchKernelGGL((grad_kernel<decltype(type), F>),
                           dim3((unsigned)tiles, (unsigned)(a.seg.adapters * a.splits), (unsigned)ceil_div(a.r, 16 * F)), dim3(256), 0, s,
                           a);
        return hipGetLastError();
    };
    auto sized = [&](auto type) {
        return a.r <= 16 ? go(type, std::integral_constant<int, 1>{})
                         : a.r <= 32 ? go(type, std::integral_constant<int, 2>{}) : go(type, std::integral_constant<int, 4>{});
    };
    const hipError_t e = dtype == ZI_F16 ? sized(f16_t{}) : sized(bf16_t{});
    if (e != hipSuccess || a.splits == 1) return e;
    const int64_t n = (int64_t)a.seg.adapters * a.r;
    return sum_parts(a.of[0].part, a.splits, n * a.of[0].K, a.of[0].G, n * a.of[1].K, a.of[1].G, a.accumulate, s);
}

bool aligned(const void *p, uint64_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

zi_status check(const zi_adapters *p) {
    if (!p) return fail(ZI_ERR_ARG, "adapters is NULL");
    // a workgroup a row, and a launch's threads are a 32-bit number
    if (p->T < 0 || p->T > (1 << 23)) return fail(ZI_ERR_SHAPE, "T = %lld: 0 .. 2^23 rows", (long long)p->T);
    if (p->K < 8 || p->M < 8 || p->K % 8 || p->M % 8 || p->K > kGroupLd || p->M > kGroupLd)
        return fail(ZI_ERR_SHAPE, "K = %lld, M = %lld: multiples of 8 up to 2^20", (long long)p->K, (long long)p->M);
    if (p->N < 1 || p->N > 65535) return fail(ZI_ERR_SHAPE, "N = %d: 1 .. 65535 adapters", p->N);
    if (p->r < 1 || p->r > kMostRank) return fail(ZI_ERR_SHAPE, "r = %d: 1 .. %d", p->r, kMostRank);
    if (p->S < 0 || p->S > (1 << 23)) return fail(ZI_ERR_SHAPE, "S = %d: 0 .. 2^23 segments", p->S);
    const int64_t lds[5] = {p->ldx, p->lddx, p->lddx0, p->ldy, p->ldy0};
    for (int i = 0; i < 5; ++i)
        if (lds[i] < 0 || lds[i] % 8 || lds[i] > kGroupLd || (lds[i] && lds[i] < (i < 3 ? p->K : p->M)))
            return fail(ZI_ERR_SHAPE, "row strides are multiples of 8, at least a row and up to 2^20");
    if (p->dtype != ZI_F16 && p->dtype != ZI_BF16) return fail(ZI_ERR_ARG, "dtype %d: fp16 or bf16", p->dtype);
    if (p->out_dtype != p->dtype && p->out_dtype != ZI_F32) return fail(ZI_ERR_ARG, "out_dtype %d: dtype or fp32", p->out_dtype);
    return ZI_OK;
}

zi_status check_work(uint64_t need, const void *workspace, uint64_t bytes) {
    if (!workspace || bytes < need)
        return fail(ZI_ERR_BUDGET, "the workspace holds %llu B, the adapters need %llu", (unsigned long long)(workspace ? bytes : 0),
                    (unsigned long long)need);
    if (!aligned(workspace, 256)) return fail(ZI_ERR_ALIGN, "the workspace is not 256-byte aligned");
    return ZI_OK;
}

Segments segments_of(const zi_adapters *p, const int32_t *offsets, const int32_t *ids) {
    return {offsets, ids, p->S, p->N, (int32_t)p->T};
}

}  // namespace
}  // namespace zi

using namespace zi;

extern "C" uint64_t zi_adapters_fwd_bytes(int64_t T, int32_t r) { return T < 1 || r < 1 ? 0 : parts_bytes(T, r) + u_bytes(T, r); }

extern "C" zi_status zi_adapters_fwd(const zi_adapters *p, const void *X, const void *A, const void *B, const int32_t *offsets,
                                     const int32_t *ids, const float *scales, const void *Y0, void *Y, float *U, void *workspace,
                                     uint64_t workspace_bytes, void *stream) {
    clear_error();
    zi_status st = check(p);
    if (st != ZI_OK || p->T == 0) return st;
    if (!X || !A || !B || !offsets || !scales || !Y || (p->S > 0 && !ids))
        return fail(ZI_ERR_ARG, "X, A, B, offsets, ids, scales and Y are required");
    if (!aligned(X, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(Y0, 16) || !aligned(Y, 16) || !aligned(offsets, 4) ||
        !aligned(ids, 4) || !aligned(scales, 4) || !aligned(U, 4))
        return fail(ZI_ERR_ALIGN, "a matrix is not 16-byte aligned, or a vector not to its element");
    if (Y0 == Y && (p->ldy0 ? p->ldy0 : p->M) != (p->ldy ? p->ldy : p->M)) return fail(ZI_ERR_SHAPE, "Y is Y0, with another row stride");
    if ((st = check_work(zi_adapters_fwd_bytes(p->T, p->r), workspace, workspace_bytes)) != ZI_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t S = max64(p->S, 1), parts = parts_of(p->T, S, p->K);
    char *work = static_cast<char *>(workspace);
    float *parted = reinterpret_cast<float *>(work), *u = U ? U : reinterpret_cast<float *>(work + parts_bytes(p->T, p->r));
    ShrinkArgs a = {};
    a.X = static_cast<const uint16_t *>(X);
    a.A = static_cast<const uint16_t *>(A);
    a.ldx = p->ldx ? p->ldx : p->K;
    a.U = parts > 1 ? parted : u;
    a.seg = segments_of(p, offsets, ids);
    a.K = (int32_t)p->K;
    a.r = p->r;
    a.block = block_of(p->T, S);
    a.parts = (int32_t)parts;
    const bool rows = a.block == 1;  // a workgroup of expand a row, which adds the parts
    hipError_t e = shrink(p->dtype, a, s);
    if (e == hipSuccess && parts > 1 && !rows) e = sum_parts(parted, parts, p->T * p->r, u, 0, nullptr, 0, s);
    if (e == hipSuccess) {
        ExpandArgs b = {};
        b.U = rows ? a.U : u;
        b.U_out = rows && parts > 1 ? U : nullptr;
        b.B = static_cast<const uint16_t *>(B);
        b.scales = scales;
        b.Y0 = Y0;
        b.Y = Y;
        b.ldy = p->ldy ? p->ldy : p->M;
        b.ldy0 = p->ldy0 ? p->ldy0 : p->M;
        b.seg = a.seg;
        b.M = (int32_t)p->M;
        b.r = p->r;
        b.parts = rows ? (int32_t)parts : 1;
        b.same = Y0 == Y;
        e = expand(p->dtype, p->out_dtype, b, rows, s);
    }
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "adapters forward: %s", hipGetErrorString(e));
    return ZI_OK;
}

extern "C" uint64_t zi_adapters_bwd_bytes(int64_t T, int32_t r) {
    return T < 1 || r < 1 ? 0 : parts_bytes(T, r) + u_bytes(T, r) + part_bytes(r);
}

extern "C" zi_status zi_adapters_bwd(const zi_adapters *p, const void *X, const void *dY, const float *U, const void *A, const void *B,
                                     const int32_t *offsets, const int32_t *ids, const float *scales, const void *dX0, void *dX,
                                     float *dA, float *dB, void *workspace, uint64_t workspace_bytes, void *stream) {
    clear_error();
    zi_status st = check(p);
    if (st != ZI_OK) return st;
    if (!dA || !dB) return fail(ZI_ERR_ARG, "dA and dB are required");
    if (p->T > 0 && (!X || !dY || !U || !A || !B || !offsets || !scales || (p->S > 0 && !ids)))
        return fail(ZI_ERR_ARG, "X, dY, U, A, B, offsets, ids and scales are required");
    if (dX0 && !dX) return fail(ZI_ERR_ARG, "dX0 without dX");
    if (!aligned(X, 16) || !aligned(dY, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(dX0, 16) || !aligned(dX, 16) ||
        !aligned(dA, 16) || !aligned(dB, 16) || !aligned(offsets, 4) || !aligned(ids, 4) || !aligned(scales, 4) || !aligned(U, 4))
        return fail(ZI_ERR_ALIGN, "a matrix is not 16-byte aligned, or a vector not to its element");
    if (dX && dX0 == dX && (p->lddx0 ? p->lddx0 : p->K) != (p->lddx ? p->lddx : p->K))
        return fail(ZI_ERR_SHAPE, "dX is dX0, with another row stride");
    if (p->T > 0 && (st = check_work(zi_adapters_bwd_bytes(p->T, p->r), workspace, workspace_bytes)) != ZI_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t S = max64(p->S, 1);
    char *work = static_cast<char *>(workspace);
    float *parted = reinterpret_cast<float *>(work), *dU = reinterpret_cast<float *>(work + parts_bytes(p->T, p->r));
    float *part = reinterpret_cast<float *>(work + parts_bytes(p->T, p->r) + u_bytes(p->T, p->r));
    const Segments seg = segments_of(p, offsets, ids);
    hipError_t e = hipSuccess;
    if (p->T > 0) {
        const int64_t parts = parts_of(p->T, S, p->M);
        ShrinkArgs a = {};
        a.X = static_cast<const uint16_t *>(dY);
        a.A = static_cast<const uint16_t *>(B);
        a.ldx = p->ldy ? p->ldy : p->M;
        a.scales = scales;
        a.U = parts == 1 ? dU : parted;
        a.seg = seg;
        a.K = (int32_t)p->M;
        a.r = p->r;
        a.block = block_of(p->T, S);
        a.parts = (int32_t)parts;
        e = shrink(p->dtype, a, s);
        if (e == hipSuccess && parts > 1) e = sum_parts(parted, parts, p->T * p->r, dU, 0, nullptr, 0, s);
        if (e == hipSuccess && dX) {
            ExpandArgs b = {};
            b.U = dU;
            b.B = static_cast<const uint16_t *>(A);
            b.Y0 = dX0;
            b.Y = dX;
            b.ldy = p->lddx ? p->lddx : p->K;
            b.ldy0 = p->lddx0 ? p->lddx0 : p->K;
            b.seg = seg;
            b.M = (int32_t)p->K;
            b.r = p->r;
            b.parts = 1;
            b.same = dX0 == dX;
            e = expand(p->dtype, p->out_dtype, b, a.block == 1, s);
        }
    }
    if (e == hipSuccess && !(p->T == 0 && p->accumulate)) {
        const int64_t tiles0 = ceil_div(p->K, 128), tiles = tiles0 + ceil_div(p->M, 128);
        GradArgs a = {};
        a.of[0] = {dU, static_cast<const uint16_t *>(X), p->ldx ? p->ldx : p->K, nullptr, dA, part, (int32_t)p->K};
        a.of[1] = {U, static_cast<const uint16_t *>(dY), p->ldy ? p->ldy : p->M, p->T == 0 ? nullptr : scales, dB,
                   part + (int64_t)p->N * p->r * p->K, (int32_t)p->M};
        a.part_split = (int64_t)p->N * p->r * (p->K + p->M);
        a.seg = seg;
        if (p->T == 0) a.seg.count = 0;  // zeros
        a.tiles0 = (int32_t)tiles0;
        a.r = p->r;
        a.splits = (int32_t)splits_of(p->T, p->N, tiles);
        a.accumulate = p->accumulate;
        e = grad(p->dtype, a, tiles, s);
    }
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "adapters backward: %s", hipGetErrorString(e));
    return ZI_OK;
}
