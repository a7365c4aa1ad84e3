// zi_orth.hip -- orthogonalising an update by Newton-Schulz products.
//
// X_0 = G / (|G|_F + eps), with the shorter side of G as rows (m x k, m <= k);
// a step is
//   A = X X^T,   X <- a X + (b A + c A^2) X,
// an odd polynomial of X's singular values, which drives them towards one.
//
// Three products a step, each one launch of the MFMA kernel (zi_orth_gemm.hip)
// with fp16 operands and fp32 sums: A and A^2 are symmetric, so only their tiles on
// and below the diagonal are formed (2 m^2 k + m^2 k + m^3 operations a step in
// place of 4 m^2 k + 2 m^3).
//
// Precision.  A step multiplies small singular values by a = 3.4, five steps by
// nearly 500, and with them whatever rounding put beside them.  So X, which the
// step carries over by a X, is held in two fp16 planes (hi + lo, 22 bits), and
// only the products' operands are rounded to 11 bits: there a rounding meets X
// through b A + c A^2, which vanishes where X is small.  The diagonals of A and
// of b A + c A^2, which hold most of their norm, and A's linear term stay in
// fp32.  That is so only while all of b A + c A^2 multiplies the same values: if
// its diagonal alone multiplied X and the rest X's high plane, what that plane
// lacks would be left over in every direction, also in those that X does not
// have, and be enlarged there (a rank-one 9 x 16 came out 4 % off).  Where at most one
// step follows, that weighs less than what the diagonal gains by both planes
// (full rank, 1001 x 1531, the same arithmetic on the CPU: 6e-4 for 9e-4), so it
// multiplies them in the last two, and always where X is a single row, whose
// polynomial is a number.
// fp16 has no step below 2^-24, so the low plane holds what it should only of
// values well above 2^-13, and X's are about 1 / sqrt(M K) or, where |G| is
// below eps, far less.  The planes are therefore X times a power of two: G's
// own for X_0, with |G| then in [2^14, 2^15), the rest of the normalisation
// being a factor in fp32; later the one that takes the largest singular value
// that X can have into [2^14, 2^15) (Bound), which no element passes.  The
// epilogues undo it; a power of two rounds nothing.  (Unscaled, a rank-one
// 2048 x 8192 came out 1.3 % off past bf16's rounding, and |G| = 1e-12 with
// eps = 1e-7 65 %; so 3e-6 and 4e-12.)
//
// What it takes.  32768 x 8192 in bf16: 28 to 29 ms, of which a step's A is 1.56 ms
// (1450 TFLOP/s on the tiles formed, the matrix cores busy 0.84 of the time),
// b A + c A^2 0.49 ms, and the product with X 3.56 ms (1235 TFLOP/s, busy 0.66:
// each tile's planes are read and written after its last multiplication).  Small
// matrices are bound by their seventeen launches: 512 x 512 takes 122 us, seven
// a launch, of which four to five pass between any two launches on a stream.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/zi.h"
#include "zi_host.h"
#include "zi_internal.h"
#include "zi_vec.h"

namespace {

using namespace zi;

constexpr int kSums = 1024;      // workgroups that sum the squares of G

int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }
int64_t min64(int64_t x, int64_t y) { return x < y ? x : y; }
int64_t max64(int64_t x, int64_t y) { return x > y ? x : y; }

// Sums of squares of G, in fp64: fp32's range would end at elements of 1e19.
template <typename T>
__global__ __launch_bounds__(256) void squares_kernel(const T *G, int64_t M, int64_t K, int64_t ld, double *sums) {
    __shared__ double part[4];
    double s = 0;
    const int64_t vecs = (K + 7) / 8, n = M * vecs;
    for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < n; j += (int64_t)kSums * 256) {
        const int64_t r = j / vecs, i = (j - r * vecs) * 8;
        float v[8];
        load_n(G + r * ld + i, K - i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += (double)v[e] * (double)v[e];
    }
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) sums[blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// The largest |p(s)|, p(s) = a s + b s^3 + c s^5, over 0 <= s <= u: at u or where
// p' is zero.
struct Bound {
    double a, b, c;
    double at[2], peak[2];  // the positive zeros of p' (infinite: none), and |p| there
    __host__ __device__ double p(double s) const { return fabs(s * (a + s * s * (b + s * s * c))); }
    __device__ double operator()(double u) const {
        double most = p(u);
        for (int k = 0; k < 2; ++k)
            if (at[k] <= u) most = fmax(most, peak[k]);
        return most;
    }
};

constexpr int kMostSteps = 100;

// The factors of every step: factor[2 j], by which the planes of X_j have to be
// multiplied to give X_j, and factor[2 j + 1], by which a step's result in terms
// of them, to give the planes of X_{j+1} (after the last step X itself).  The
// power of two of X_{j+1}'s planes is at least one, so that a polynomial
// whose bound grows without end loses nothing by it.
__device__ __forceinline__ void write_factors(const Bound &bound, int steps, double norm, double eps, int e2, float *factor) {
    // (norm 0: all planes are zero, and times zero they stay so, also without eps)
    double in = norm == 0 ? 0 : 1.0 / ldexp(norm + eps, e2), most = norm == 0 ? 0 : norm / (norm + eps);
    for (int j = 0; j < steps; ++j) {
        most = bound(most);
        int e = 0;  // (NaN and infinities: 0)
        if (most < 32768) {
            (void)frexp(most, &e);
            e = min(15 - e, 120);
        }
        if (j + 1 == steps) e = 0;
        factor[2 * j] = (float)in;
        factor[2 * j + 1] = (float)ldexp(in, e);
        in = ldexp(1.0, -e);
    }
}

// The planes of X_0, 64 x 64 elements a workgroup (TR: X is G transposed), and
// zeros up to the padded extents; workgroup (0, 0) also writes the steps'
// factors and clears the counters of split tiles.
template <typename T, bool TR>
__global__ __launch_bounds__(256) void planes_kernel(const T *G, int64_t M, int64_t K, int64_t ldg, const double *sums,
                                                     float eps, uint16_t *hi, uint16_t *lo, int64_t ld, Bound bound,
                                                     int32_t steps, float *factor, uint32_t *cnt) {
    __shared__ double part[4];
    __shared__ float tile[64][65];
    double s = 0;
    for (int j = threadIdx.x; j < kSums; j += 256) s += sums[j];
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) s += __shfl_xor(s, m, 64);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    // G's rows and columns that this tile holds
    const int64_t x0 = (int64_t)blockIdx.x * 64, y0 = (int64_t)blockIdx.y * 64;  // X's column, row
    const int64_t r0 = TR ? x0 : y0, c0 = TR ? y0 : x0;
    const int row = threadIdx.x >> 3, col = (threadIdx.x & 7) * 8;
#pragma unroll
    for (int h = 0; h < 64; h += 32) {
        float v[8];
        const int64_t r = r0 + row + h;
        load_n(G + r * ldg + c0 + col, r < M ? K - c0 - col : 0, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) tile[row + h][col + e] = v[e];
    }
    __syncthreads();
    const double norm = sqrt(part[0] + part[1] + part[2] + part[3]);
    int e2 = 0;  // norm 2^e2 in [2^14, 2^15)
    if (norm > 0 && norm < INFINITY) {
        (void)frexp(norm, &e2);
        e2 = 15 - e2;
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        if (threadIdx.x == 0) write_factors(bound, steps, norm, (double)eps, e2, factor);
        for (int j = threadIdx.x; j < kOrthSplits; j += 256) cnt[j] = 0;
    }
#pragma unroll
    for (int h = 0; h < 64; h += 32) {
        uint16_t a[8], b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = ldexpf(TR ? tile[col + e][row + h] : tile[row + h][col + e], e2);
            a[e] = __builtin_bit_cast(uint16_t, (f16_t)x);
            b[e] = __builtin_bit_cast(uint16_t, (f16_t)(x - to_f32<f16_t>(a[e])));
        }
        const int64_t at = (y0 + row + h) * ld + x0 + col;
        u16x8_u va, vb;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            va[e] = a[e];
            vb[e] = b[e];
        }
        *reinterpret_cast<u16x8_u *>(hi + at) = va;
        *reinterpret_cast<u16x8_u *>(lo + at) = vb;
    }
}

// ---- host ---------------------------------------------------------------------------

// Sizes and the workspace of one orthogonalisation.
struct Work {
    int64_t m, k, mp, kp;  // the shorter and the longer side, and padded to 64
    uint64_t hi[2], lo, o16, b16, o32, diag, bdiag, sums, factor, cnt, part, bytes;
};

// The side of the products' tiles: 256 where the triangle has at least one tile
// for each compute unit; else 128, two workgroups a unit, or, for narrow
// matrices and those whose m x k product fills no round of those, 64, four a
// unit.  With tiles of 64 and of 128: 1024 x 1536 203 and 313 us, 1536 x 6144
// 622 and 655, 2048 x 2048 417 and 561; 2048 x 8192 1110 and 958, 3008 x 3008
// 1027 and 912.
int tile_of(int64_t mp, int64_t kp) {
    const int64_t n = (mp + 255) / 256;
    if (n * (n + 1) / 2 >= kOrthUnits) return 256;
    return mp <= 1536 || ((mp + 127) / 128) * ((kp + 127) / 128) <= 2 * kOrthUnits ? 64 : 128;
}

Work work_of(int64_t M, int64_t K) {
    Work w;
    w.m = min64(M, K);
    w.k = max64(M, K);
    w.mp = up(w.m, 64);
    w.kp = up(w.k, 64);
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const uint64_t x = (uint64_t)w.mp * w.kp * 2, a = (uint64_t)w.mp * w.mp * 2;
    w.hi[0] = take(x);
    w.hi[1] = take(x);
    w.lo = take(x);
    w.o16 = take(a);
    w.b16 = take(a);
    w.o32 = take(2 * a);
    w.diag = take((uint64_t)w.mp * 4);
    w.bdiag = take((uint64_t)w.mp * 4);
    w.sums = take(kSums * 8);
    w.factor = take(kMostSteps * 8);
    w.cnt = take(kOrthSplits * 4);
    w.part = take(orth_split_bytes(tile_of(w.mp, w.kp)));
    w.bytes = at;
    return w;
}

Bound bound_of(const zi_orth &o) {
    Bound f{o.a, o.b, o.c, {INFINITY, INFINITY}, {}};
    // p'(s) = a + 3 b t + 5 c t^2, t = s^2
    double t[2] = {-1, -1};
    if (f.c != 0) {
        const double mid = -0.3 * f.b / f.c, both = 0.2 * f.a / f.c, wide = mid * mid - both;  // both: t0 t1
        if (wide >= 0) {
            t[0] = mid + copysign(sqrt(wide), mid);  // the larger one: no digits cancel
            if (t[0] != 0) t[1] = both / t[0];
        }
    } else if (f.b != 0) {
        t[0] = -f.a / (3 * f.b);
    }
    for (int k = 0; k < 2; ++k)
        if (t[k] > 0) {
            f.at[k] = sqrt(t[k]);
            f.peak[k] = f.p(f.at[k]);
        }
    return f;
}

template <typename T>
hipError_t run(const zi_orth *o, const void *G, void *O, char *base, hipStream_t s) {
    const Work w = work_of(o->M, o->K);
    const int64_t ldg = o->ldg ? o->ldg : o->K, ldo = o->ldo ? o->ldo : o->K;
    const bool tr = o->M > o->K;
    const int tile = tile_of(w.mp, w.kp);
    double *sums = reinterpret_cast<double *>(base + w.sums);
    float *factor = reinterpret_cast<float *>(base + w.factor);
    uint16_t *hi[2] = {reinterpret_cast<uint16_t *>(base + w.hi[0]), reinterpret_cast<uint16_t *>(base + w.hi[1])};
    uint16_t *lo = reinterpret_cast<uint16_t *>(base + w.lo);
    uint32_t *cnt = reinterpret_cast<uint32_t *>(base + w.cnt);
    hipError_t e;
    hipLaunchKernelGGL(squares_kernel<T>, dim3(kSums), dim3(256), 0, s, static_cast<const T *>(G), o->M, o->K, ldg, sums);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const dim3 g((unsigned)(w.kp / 64), (unsigned)(w.mp / 64));
    if (tr)
        hipLaunchKernelGGL((planes_kernel<T, true>), g, dim3(256), 0, s, static_cast<const T *>(G), o->M, o->K, ldg, sums,
                           o->eps, hi[0], lo, w.kp, bound_of(*o), o->steps, factor, cnt);
    else
        hipLaunchKernelGGL((planes_kernel<T, false>), g, dim3(256), 0, s, static_cast<const T *>(G), o->M, o->K, ldg, sums,
                           o->eps, hi[0], lo, w.kp, bound_of(*o), o->steps, factor, cnt);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    OrthArgs c{};
    c.ca = o->a;
    c.cb = o->b;
    c.cc = o->c;
    c.diag = reinterpret_cast<float *>(base + w.diag);
    c.bdiag = reinterpret_cast<float *>(base + w.bdiag);
    c.o32 = reinterpret_cast<float *>(base + w.o32);
    c.split_part = reinterpret_cast<float *>(base + w.part);
    c.split_cnt = cnt;
    c.rows = w.mp;
    for (int step = 0; step < o->steps; ++step) {
        uint16_t *x = hi[step & 1];
        OrthArgs a = c;  // A = X X^T
        a.scale = factor + 2 * step;
        a.Q = a.P = x;
        a.ldq = a.ldp = w.kp;
        a.C = base + w.o16;
        a.ldc = w.mp;
        a.cols = w.mp;
        a.red = w.kp;
        if ((e = launch_orth(OrthOp::Gram, tile, a, s)) != hipSuccess) return e;
        a = c;  // b A + c A^2
        a.Q = a.P = base + w.o16;
        a.ldq = a.ldp = w.mp;
        a.C = base + w.b16;
        a.ldc = w.mp;
        a.cols = w.mp;
        a.red = w.mp;
        if ((e = launch_orth(OrthOp::Poly, tile, a, s)) != hipSuccess) return e;
        a = c;  // a X + (b A + c A^2) X
        a.scale = factor + 2 * step + 1;
        a.Q = a.hi = x;
        a.ldq = w.kp;
        a.P = base + w.b16;
        a.ldp = w.mp;
        a.lo = lo;
        a.diag_x = w.m == 1 || step + 2 >= o->steps;
        a.ldc = w.kp;
        a.cols = w.kp;
        a.red = w.mp;
        if (step + 1 < o->steps) {
            a.hi_out = hi[(step + 1) & 1];
        } else {
            a.out = static_cast<uint16_t *>(O);
            a.out_p = w.m;
            a.out_q = w.k;
            a.out_ld = ldo;
            a.out_t = tr;
        }
        if ((e = launch_orth(OrthOp::Apply, tile, a, s)) != hipSuccess) return e;
    }
    return hipSuccess;
}

bool aligned(const void *p, uint64_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

}  // namespace

extern "C" uint64_t zi_orthogonalize_bytes(int64_t M, int64_t K) {
    if (M < 1 || K < 1 || M > ZI_ORTH_MOST || K > ZI_ORTH_MOST) return 0;
    return work_of(M, K).bytes;
}

extern "C" zi_status zi_orthogonalize(const zi_orth *o, const void *G, void *O, void *workspace,
                                      uint64_t workspace_bytes, void *stream) {
    clear_error();
    if (!o) return fail(ZI_ERR_ARG, "orth is NULL");
    if (o->M < 1 || o->K < 1 || o->M > ZI_ORTH_MOST || o->K > ZI_ORTH_MOST)
        return fail(ZI_ERR_SHAPE, "M = %lld, K = %lld: 1 .. %d each", (long long)o->M, (long long)o->K, ZI_ORTH_MOST);
    if ((o->ldg != 0 && o->ldg < o->K) || (o->ldo != 0 && o->ldo < o->K))
        return fail(ZI_ERR_SHAPE, "a row stride is less than K");
    if (o->dtype != ZI_F16 && o->dtype != ZI_BF16 && o->dtype != ZI_F32)
        return fail(ZI_ERR_ARG, "unknown dtype %d", o->dtype);
    if (o->steps < 1 || o->steps > kMostSteps) return fail(ZI_ERR_ARG, "steps = %d: 1 .. %d", o->steps, kMostSteps);
    if (!isfinite(o->a) || !isfinite(o->b) || !isfinite(o->c) || !(o->eps >= 0.f) || !isfinite(o->eps))
        return fail(ZI_ERR_ARG, "a, b, c and eps must be finite, and eps not negative");
    if (!G || !O) return fail(ZI_ERR_ARG, "G and O are required");
    if (!aligned(G, o->dtype == ZI_F32 ? 4 : 2) || !aligned(O, 2))
        return fail(ZI_ERR_ALIGN, "a pointer is not aligned to its element");
    const uint64_t need = work_of(o->M, o->K).bytes;
    if (!workspace || workspace_bytes < need)
        return fail(ZI_ERR_BUDGET, "the workspace holds %llu B, %llu are needed",
                    (unsigned long long)(workspace ? workspace_bytes : 0), (unsigned long long)need);
    if (!aligned(workspace, 256)) return fail(ZI_ERR_ALIGN, "the workspace is not 256-byte aligned");
    hipStream_t s = static_cast<hipStream_t>(stream);
    char *base = static_cast<char *>(workspace);
    const hipError_t e = o->dtype == ZI_F32   ? run<float>(o, G, O, base, s)
                         : o->dtype == ZI_F16 ? run<f16_t>(o, G, O, base, s)
                                              : run<bf16_t>(o, G, O, base, s);
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "orthogonalisation: %s", hipGetErrorString(e));
    return ZI_OK;
}
