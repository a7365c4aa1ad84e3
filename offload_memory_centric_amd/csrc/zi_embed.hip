// zi_embed.hip -- token embedding, forward and gradient.
//
// Forward:   X[t] = RNE(scale W[id_t])
// Gradient:  dW[v] (+)= scale * sum of dX[t] over the tokens t with id_t = v
// An id outside [0, V) marks padding: its row of X is zero and it has no
// gradient.
//
// The gradient has no atomics on values, so that it is the same every time.
// The tokens are sorted by id (ties by position) and the sorted list is cut
// into chunks of kChunk tokens.  A run of equal ids that lies in one chunk is
// summed straight into its row of dW.  A run that crosses a chunk's border, such
// as a frequent token's, is summed piece by piece, one piece a chunk, into the
// workspace, and its pieces are then added in order.  Rows without a token are
// written as zero by the same launch.  Sums are held in fp32 and rounded once.
//
// The sort: a workgroup ranks 256 keys of a tile of kTile by counting the
// tile's smaller ones; kFan sorted lists at a time are then merged, the place
// of a key being its place in its own list plus the number of keys before it in
// every other one (binary searches).  32768 tokens take one merge.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/zi.h"
#include "zi_host.h"
#include "zi_vec.h"

namespace {

using namespace zi;

constexpr int kChunk = 64;   // sorted tokens of a chunk
constexpr int kTile = 1024;  // tokens that the first step sorts together
constexpr int kFan = 32;     // lists that one merge joins

constexpr int64_t kMostGroups = 1 << 20;  // workgroups along one side of a grid (a side ends below 2^32 threads)

int64_t min64(int64_t x, int64_t y) { return x < y ? x : y; }
int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
uint64_t up256(uint64_t x) { return (x + 255) / 256 * 256; }

// The id at position t, or V (past every row) for padding.
__device__ __forceinline__ uint32_t key_at(const void *ids, bool wide, int64_t t, int64_t V) {
    const int64_t id = wide ? static_cast<const int64_t *>(ids)[t] : (int64_t) static_cast<const int32_t *>(ids)[t];
    return (uint32_t)(id < 0 || id >= V ? V : id);
}

// L lanes a token, 256 / L tokens a workgroup; blockIdx.y: a span of columns.
constexpr int kSpan = 8;  // vectors a lane takes of one token
template <typename WT, typename XT, int L>
__global__ __launch_bounds__(256) void embed_fwd_kernel(const void *ids, int32_t wide, int64_t T, int64_t V, int64_t D,
                                                        const WT *W, int64_t ldw, float scale, XT *X, int64_t ldx) {
    const int64_t base = ((int64_t)blockIdx.y * kSpan * L + threadIdx.x % L) * 8;
    for (int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L; t < T; t += (int64_t)gridDim.x * (256 / L)) {
        const uint32_t v = key_at(ids, wide, t, V);
        const WT *w = W + (int64_t)v * ldw;
        XT *x = X + t * ldx;
        float r[kSpan][8];
#pragma unroll
        for (int c = 0; c < kSpan; ++c) {
            const int64_t i = base + c * L * 8;
            load_n(w + i, v < V ? D - i : 0, r[c]);
        }
#pragma unroll
        for (int c = 0; c < kSpan; ++c) {
            const int64_t i = base + c * L * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) r[c][e] *= scale;
            if (D - i >= 8) stream8(x + i, r[c]);
            else store_n(x + i, D - i, r[c]);
        }
    }
}

// ---- the sort -----------------------------------------------------------------------

// The rank of 256 keys (blockIdx.y) of tile blockIdx.x among the tile's.
__global__ __launch_bounds__(256) void sort_tile_kernel(const void *ids, int32_t wide, int64_t T, int64_t V,
                                                        uint32_t *keys, int32_t *order) {
    __shared__ uint32_t k[kTile];
    const int64_t base = (int64_t)blockIdx.x * kTile;
    const int n = (int)min((int64_t)kTile, T - base);
    for (int j = threadIdx.x; j < kTile; j += 256) k[j] = j < n ? key_at(ids, wide, base + j, V) : 0xffffffffu;
    __syncthreads();
    const int i = blockIdx.y * 256 + threadIdx.x;
    const int w0 = __builtin_amdgcn_readfirstlane(i & ~63);  // the wave's own 64 positions
    const uint32_t mine = k[i];
    int rank = 0;
    for (int j = 0; j < w0; ++j) rank += k[j] <= mine;  // equal keys before come first
    for (int j = w0; j < w0 + 64; ++j) rank += k[j] < mine || (k[j] == mine && j < i);
    for (int j = w0 + 64; j < kTile; ++j) rank += k[j] < mine;
    if (i < n) {
        keys[base + rank] = mine;
        order[base + rank] = (int32_t)(base + i);
    }
}

// Keys of the sorted list [p, p + n) that come before `key` (OR_EQUAL: or equal it).
template <bool OR_EQUAL>
__device__ __forceinline__ int64_t before(const uint32_t *p, int64_t n, uint32_t key) {
    int64_t lo = 0;
    while (n > 0) {
        const int64_t half = n >> 1;
        const bool right = OR_EQUAL ? p[lo + half] <= key : p[lo + half] < key;
        lo = right ? lo + half + 1 : lo;
        n = right ? n - half - 1 : half;
    }
    return lo;
}

// Joins groups of kFan sorted lists of `len` keys each.
__global__ __launch_bounds__(256) void merge_kernel(const uint32_t *keys, const int32_t *order, uint32_t *keys_out,
                                                    int32_t *order_out, int64_t T, int64_t len) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= T) return;
    const int64_t list = i / len, first = list / kFan * kFan;
    const uint32_t key = keys[i];
    int64_t at = first * len + (i - list * len);
    for (int64_t l = first; l < first + kFan; ++l) {
        const int64_t from = l * len;
        if (from >= T) break;
        const int64_t n = min(len, T - from);
        if (l < list)
            at += before<true>(keys + from, n, key);
        else if (l > list)
            at += before<false>(keys + from, n, key);
    }
    keys_out[at] = key;
    order_out[at] = order[i];
}

// ---- the sums -----------------------------------------------------------------------

// Adds rows order[j] of dX, j in [from, to), columns [i, i + 8).
template <typename DT>
__device__ __forceinline__ void add_rows(const DT *dX, int64_t ldx, const int32_t *order, int64_t from, int64_t to,
                                         int64_t i, int64_t n, float (&s)[8]) {
    for (int64_t j = from; j < to; ++j) {
        float u[8];
        load_n(dX + (int64_t)order[j] * ldx + i, n, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += u[e];
    }
}

// Chunk blockIdx.x of the sorted tokens: notes where each run begins and ends
// (first[v], last[v]), and sums the pieces of the runs that cross its borders:
// of the one that comes in from the left into slot 0, of the one that goes on
// to the right (if it begins here) into slot 1.
template <typename DT>
__global__ __launch_bounds__(256) void piece_kernel(const uint32_t *keys, const int32_t *order, int64_t T, int64_t V,
                                                    const DT *dX, int64_t ldx, int64_t D, int32_t *first,
                                                    int32_t *last, float *pieces) {
    const int64_t a = (int64_t)blockIdx.x * kChunk, b = min(a + kChunk, T);
    const uint32_t ka = keys[a], kb = keys[b - 1];
    if (blockIdx.y == 0 && threadIdx.x < b - a) {
        const int64_t j = a + threadIdx.x;
        const uint32_t k = keys[j];
        if (k < V) {
            if (j == 0 || keys[j - 1] != k) first[k] = (int32_t)j;
            if (j == T - 1 || keys[j + 1] != k) last[k] = (int32_t)j;
        }
    }
    const bool in = a > 0 && keys[a - 1] == ka && ka < V;
    const bool on = b < T && keys[b] == kb && kb < V;
    const int64_t i = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 8;
    if (i >= D) return;
    if (in || (on && ka == kb)) {
        float s[8] = {};
        int64_t to = a;
        while (to < b && keys[to] == ka) ++to;
        add_rows(dX, ldx, order, a, to, i, D - i, s);
        store_n(pieces + (2 * (int64_t)blockIdx.x) * D + i, D - i, s);
    }
    if (on && ka != kb) {
        float s[8] = {};
        int64_t from = b;
        while (keys[from - 1] == kb) --from;
        add_rows(dX, ldx, order, from, b, i, D - i, s);
        store_n(pieces + (2 * (int64_t)blockIdx.x + 1) * D + i, D - i, s);
    }
}

// Row v of dW.  first[v] means something only where v has tokens; the entry of
// any other row is whatever the workspace held, so it is checked against the
// sorted keys, which are all written: v has tokens exactly if its entry is a
// place in the list that holds v and is the first one to do so.
template <typename DT, typename WT>
__global__ __launch_bounds__(256) void row_kernel(const uint32_t *keys, const int32_t *order, int64_t T, int64_t V,
                                                  const DT *dX, int64_t ldx, int64_t D, const int32_t *first,
                                                  const int32_t *last, const float *pieces, float scale,
                                                  int32_t accumulate, WT *dW, int64_t ldw) {
    const int64_t i = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 8;
    if (i >= D) return;
    for (int64_t v = blockIdx.x; v < V; v += gridDim.x) {
        WT *w = dW + v * ldw + i;
        const int64_t f = T > 0 ? first[v] : -1;
        const bool has = f >= 0 && f < T && keys[f] == (uint32_t)v && (f == 0 || keys[f - 1] != (uint32_t)v);
        float s[8] = {};
        if (has) {
            const int64_t l = last[v];
            const int64_t ca = f / kChunk, cb = l / kChunk;
            if (ca == cb) {
                add_rows(dX, ldx, order, f, l + 1, i, D - i, s);
            } else {
                // the first piece is slot 0 if the run begins its chunk, else slot 1
                for (int64_t c = ca; c <= cb; ++c) {
                    float u[8];
                    const int64_t slot = 2 * c + (c == ca && f > c * kChunk ? 1 : 0);
                    load_n(pieces + slot * D + i, D - i, u);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s[e] += u[e];
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] *= scale;
        }
        if (accumulate) {
            if (!has) continue;
            float u[8];
            load_n(w, D - i, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += u[e];
        }
        store_n(w, D - i, s);
    }
}

// ---- host ---------------------------------------------------------------------------

// The workspace of a gradient: two sets of keys and positions (the sort goes
// from one to the other), the runs' ends, the pieces.
struct Work {
    uint64_t keys[2], order[2], first, last, pieces, bytes;
};
Work work_of(int64_t T, int64_t V, int64_t D) {
    Work w;
    uint64_t at = 0;
    for (int k = 0; k < 2; ++k) {
        w.keys[k] = at;
        at += up256((uint64_t)T * 4);
        w.order[k] = at;
        at += up256((uint64_t)T * 4);
    }
    w.first = at;
    at += up256((uint64_t)V * 4);
    w.last = at;
    at += up256((uint64_t)V * 4);
    w.pieces = at;
    at += up256((uint64_t)ceil_div(T, kChunk) * 2 * (uint64_t)D * 4);
    w.bytes = at;
    return w;
}

template <typename WT, typename XT>
hipError_t run_fwd(const zi_embedding *p, const void *ids, const void *W, void *X, hipStream_t s) {
    const bool wide = p->ids64 != 0;
    const int64_t vecs = ceil_div(p->D, 8), ldw = p->ldw ? p->ldw : p->D, ldx = p->ldx ? p->ldx : p->D;
    auto go = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value;
        const dim3 g((unsigned)min64(ceil_div(p->T, 256 / L), kMostGroups), (unsigned)ceil_div(vecs, L * kSpan));
        hipLaunchKernelGGL((embed_fwd_kernel<WT, XT, L>), g, dim3(256), 0, s, ids, wide, p->T, p->V, p->D,
                           static_cast<const WT *>(W), ldw, p->scale, static_cast<XT *>(X), ldx);
        return hipGetLastError();
    };
    if (vecs <= 16) return go(std::integral_constant<int, 16>{});
    if (vecs <= 64) return go(std::integral_constant<int, 64>{});
    return go(std::integral_constant<int, 256>{});
}

template <typename DT, typename WT>
hipError_t run_bwd(const zi_embedding *p, const void *ids, const void *dX, void *dW, char *work, hipStream_t s) {
    const int64_t T = p->T, V = p->V, D = p->D;
    const int64_t ldw = p->ldw ? p->ldw : D, ldx = p->ldx ? p->ldx : D;
    const unsigned spans = (unsigned)ceil_div(D, 2048);
    const Work w = work_of(T, V, D);
    uint32_t *keys[2] = {};
    int32_t *order[2] = {}, *first = nullptr, *last = nullptr;
    float *pieces = nullptr;
    int k = 0;
    hipError_t e;
    if (T > 0) {
        for (int j = 0; j < 2; ++j) {
            keys[j] = reinterpret_cast<uint32_t *>(work + w.keys[j]);
            order[j] = reinterpret_cast<int32_t *>(work + w.order[j]);
        }
        first = reinterpret_cast<int32_t *>(work + w.first);
        last = reinterpret_cast<int32_t *>(work + w.last);
        pieces = reinterpret_cast<float *>(work + w.pieces);
        hipLaunchKernelGGL(sort_tile_kernel, dim3((unsigned)ceil_div(T, kTile), kTile / 256), dim3(256), 0, s, ids,
                           p->ids64 != 0, T, V, keys[0], order[0]);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        for (int64_t len = kTile; len < T; len *= kFan, k ^= 1) {
            hipLaunchKernelGGL(merge_kernel, dim3((unsigned)ceil_div(T, 256)), dim3(256), 0, s, keys[k], order[k],
                               keys[k ^ 1], order[k ^ 1], T, len);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
        hipLaunchKernelGGL((piece_kernel<DT>), dim3((unsigned)ceil_div(T, kChunk), spans), dim3(256), 0, s, keys[k],
                           order[k], T, V, static_cast<const DT *>(dX), ldx, D, first, last, pieces);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    hipLaunchKernelGGL((row_kernel<DT, WT>), dim3((unsigned)min64(V, kMostGroups), spans), dim3(256), 0, s, keys[k], order[k],
                       T, V, static_cast<const DT *>(dX), ldx, D, first, last, pieces, p->scale, p->accumulate,
                       static_cast<WT *>(dW), ldw);
    return hipGetLastError();
}

// f(type of W or dW, type of X or dX) for every pair.
template <typename F>
hipError_t with_types(int32_t w, int32_t x, F &&f) {
    auto second = [&](auto wt) {
        if (x == ZI_F32) return f(wt, float{});
        if (x == ZI_F16) return f(wt, f16_t{});
        return f(wt, bf16_t{});
    };
    if (w == ZI_F32) return second(float{});
    if (w == ZI_F16) return second(f16_t{});
    return second(bf16_t{});
}

bool known(int32_t d) { return d == ZI_F16 || d == ZI_BF16 || d == ZI_F32; }
bool aligned(const void *p, uint64_t to) { return ((uintptr_t)p & (to - 1)) == 0; }

zi_status check(const zi_embedding *p, const void *ids, const void *W, const void *X) {
    if (!p) return fail(ZI_ERR_ARG, "embedding is NULL");
    // a chunk's borders and a token's position are 32-bit numbers
    if (p->T < 0 || p->T > INT32_MAX - kTile) return fail(ZI_ERR_SHAPE, "T = %lld is out of range", (long long)p->T);
    if (p->V < 1 || p->V > INT32_MAX) return fail(ZI_ERR_SHAPE, "V = %lld: 1 .. 2^31 - 1 rows", (long long)p->V);
    // spans of columns are a grid's second dimension
    if (p->D < 1 || p->D > 65535 * (int64_t)2048) return fail(ZI_ERR_SHAPE, "D = %lld is out of range", (long long)p->D);
    if (!known(p->w_dtype) || !known(p->x_dtype))
        return fail(ZI_ERR_ARG, "unknown dtype (w %d, x %d)", p->w_dtype, p->x_dtype);
    if ((p->ldw != 0 && p->ldw < p->D) || (p->ldx != 0 && p->ldx < p->D))
        return fail(ZI_ERR_SHAPE, "a row stride is less than D");
    if (!isfinite(p->scale)) return fail(ZI_ERR_ARG, "scale = %g", (double)p->scale);
    if (p->T > 0 && (!ids || !X)) return fail(ZI_ERR_ARG, "the ids and the token rows are required");
    if (!W) return fail(ZI_ERR_ARG, "the table is required");
    if (!aligned(ids, p->ids64 ? 8 : 4) || !aligned(W, p->w_dtype == ZI_F32 ? 4 : 2) ||
        !aligned(X, p->x_dtype == ZI_F32 ? 4 : 2))
        return fail(ZI_ERR_ALIGN, "a pointer is not aligned to its element");
    return ZI_OK;
}

}  // namespace

extern "C" zi_status zi_embedding_fwd(const zi_embedding *p, const void *ids, const void *W, void *X, void *stream) {
    clear_error();
    const zi_status st = check(p, ids, W, X);
    if (st != ZI_OK || p->T == 0) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = with_types(p->w_dtype, p->x_dtype, [&](auto w, auto x) {
        return run_fwd<decltype(w), decltype(x)>(p, ids, W, X, s);
    });
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "embedding forward: %s", hipGetErrorString(e));
    return ZI_OK;
}

extern "C" uint64_t zi_embedding_bwd_bytes(int64_t T, int64_t V, int64_t D) {
    if (T < 1 || V < 1 || D < 1) return 0;
    return work_of(T, V, D).bytes;
}

extern "C" zi_status zi_embedding_bwd(const zi_embedding *p, const void *ids, const void *dX, void *dW,
                                      void *workspace, uint64_t workspace_bytes, void *stream) {
    clear_error();
    const zi_status st = check(p, ids, dW, dX);
    if (st != ZI_OK) return st;
    if (p->T == 0 && p->accumulate) return ZI_OK;
    const uint64_t need = zi_embedding_bwd_bytes(p->T, p->V, p->D);
    if (need && (!workspace || workspace_bytes < need))
        return fail(ZI_ERR_BUDGET, "the workspace holds %llu B, the gradient needs %llu",
                    (unsigned long long)(workspace ? workspace_bytes : 0), (unsigned long long)need);
    if (!aligned(workspace, 256)) return fail(ZI_ERR_ALIGN, "the workspace is not 256-byte aligned");
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = with_types(p->w_dtype, p->x_dtype, [&](auto w, auto x) {
        return run_bwd<decltype(x), decltype(w)>(p, ids, dX, dW, static_cast<char *>(workspace), s);
    });
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "embedding gradient: %s", hipGetErrorString(e));
    return ZI_OK;
}
