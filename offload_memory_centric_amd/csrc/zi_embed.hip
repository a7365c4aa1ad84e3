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
// written as zero.  Sums are held in fp32 and rounded once.
//
// The sort: a workgroup ranks 64 keys of a tile by counting the tile's smaller
// ones; up to 4096 tokens are one tile.  Of more, kFan sorted lists at a time
// are then merged, the place of a key being its place in its own list plus the
// number of keys before it in every other one (binary searches).  32768 tokens
// take one merge.
// What it takes.  Forward, 32768 tokens of 25600 fp16 values: 431 us, 2.18 GB at
// 5.1 TB/s.  Gradient of 32768 tokens of 8192 bf16 values in 50257 fp32 rows:
// 466 us, of which the sums and the zeros (2.15 GB) are 405, 5.3 TB/s, and the
// sort 20.  Of 2047 tokens of 512 fp32 values, 107 MB of them zeros: 30 us; the
// sort, the sums and the joins wait for latencies, the fill runs beside the sort.
// Of 262144 tokens of 1024 bf16 values 282 us: the sort 114, of which the second
// merge, whose searches are in memory, 30; of 65536 tokens 108: 31 and 6.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/zi.h"
#include "zi_host.h"
#include "zi_vec.h"

namespace {

using namespace zi;

constexpr int kChunk = 64;      // sorted tokens of a chunk, at most
constexpr int kTile = 1024;     // tokens that the first step sorts together,
constexpr int kOneTile = 4096;  // or all of them, if they are no more than this
constexpr int kFan = 32;        // lists that one merge joins

constexpr int64_t kMostGroups = 1 << 20;  // workgroups along one side of a grid (a side ends below 2^32 threads)

int64_t min64(int64_t x, int64_t y) { return x < y ? x : y; }
int64_t max64(int64_t x, int64_t y) { return x > y ? x : y; }
int64_t ceil_div(int64_t x, int64_t y) { return (x + y - 1) / y; }
uint64_t up256(uint64_t x) { return (x + 255) / 256 * 256; }

// The id, or V (past every row) for padding.
__device__ __forceinline__ uint32_t key_of(int64_t id, int64_t V) { return (uint32_t)(id < 0 || id >= V ? V : id); }

// L lanes a token, 256 / L tokens a workgroup; blockIdx.y: a span of columns.
// All of a lane's loads are in flight before its first store; X passes the
// caches, W, whose rows come again, does not.  A row's last vector is moved back
// to end with the row: the elements that it shares with the one before it are
// written twice, with one value.  (Rows of less than eight columns: TINY.)
constexpr int kSpan = 4;  // vectors a lane takes of one token (3: 1 % slower for long rows, 2: 4 %)
template <typename WT, typename XT, int L, bool TINY>
__global__ __launch_bounds__(256) void embed_fwd_kernel(const void *ids, int32_t wide, int64_t T, int64_t V, int64_t D,
                                                        const WT *__restrict__ W, int64_t ldw, float scale,
                                                        XT *__restrict__ X, int64_t ldx) {
    const int64_t base = ((int64_t)blockIdx.y * kSpan * L + threadIdx.x % L) * 8;
    for (int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L; t < T; t += (int64_t)gridDim.x * (256 / L)) {
        const uint32_t v = key_of(wide ? static_cast<const int64_t *>(ids)[t] : static_cast<const int32_t *>(ids)[t], V);
        const bool in = v < V;
        const WT *w = W + (int64_t)(in ? v : 0) * ldw;
        XT *x = X + t * ldx;
        float r[kSpan][8];
#pragma unroll
        for (int c = 0; c < kSpan; ++c) {
            const int64_t i = base + c * L * 8;
            if constexpr (TINY) load_n(w + i, D - i, r[c]);
            else load8(w + min(i, D - 8), r[c]);
        }
#pragma unroll
        for (int c = 0; c < kSpan; ++c) {
            const int64_t i = base + c * L * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) r[c][e] = in ? r[c][e] * scale : 0.f;
            if constexpr (TINY) {
                store_n(x + i, D - i, r[c]);
            } else {
                if (i < D) stream8(x + min(i, D - 8), r[c]);
            }
        }
    }
}

// ---- the sort -----------------------------------------------------------------------

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr uint32_t kNoKey = 0xffffffffu;  // past every key

// Rows of dW that are written as zero, whatever their type.
struct Fill {
    char *base;
    int64_t V, stride, bytes;  // rows; from one to the next, and of one, in bytes (even)
    int32_t rows;              // that a workgroup takes at a time
};
constexpr int kMostRows = 64;

__device__ __forceinline__ void fill_row(const Fill &f, int64_t v) {
    char *w = f.base + v * f.stride;
    for (int64_t i = threadIdx.x * 16; i + 16 <= f.bytes; i += blockDim.x * 16)
        __builtin_nontemporal_store(u32x4_u{}, reinterpret_cast<u32x4_u *>(w + i));
    const int64_t i = f.bytes / 16 * 16 + threadIdx.x * 2;
    if (i < f.bytes) *reinterpret_cast<uint16_t *>(w + i) = 0;
}

// The place of 64 keys of a tile blockIdx.x in the sorted tile: the
// number of keys that are smaller, or equal and before.  Each of 16 waves
// counts over its share of the tile, four keys a read.  Workgroups from
// `sorts` on fill all of dW, if it is filled here.
template <int TILE, typename ID>
__global__ __launch_bounds__(1024) void sort_tile_kernel(const ID *__restrict__ ids, int64_t T, int64_t V,
                                                         uint32_t *__restrict__ keys, int32_t *__restrict__ order,
                                                         int32_t sorts, int32_t per_tile, Fill fill) {
    if ((int)blockIdx.x >= sorts) {
        const int64_t first = (int64_t)(blockIdx.x - sorts) * fill.rows, step = (int64_t)(gridDim.x - sorts) * fill.rows;
        for (int64_t v0 = first; v0 < fill.V; v0 += step)
            for (int64_t v = v0; v < min(v0 + fill.rows, fill.V); ++v) fill_row(fill, v);
        return;
    }
    constexpr int SHARE = TILE / 16;
    static_assert(SHARE % 64 == 0, "the 64 keys lie in one wave's share");
    __shared__ __attribute__((aligned(16))) uint32_t k[TILE];
    __shared__ int count[16][64];
    const int64_t base = (int64_t)(blockIdx.x / per_tile) * TILE;
    const int n = (int)min((int64_t)TILE, T - base);
#pragma unroll
    for (int c = 0; c < TILE / 1024; ++c) {  // every load in flight at once
        const int j = c * 1024 + threadIdx.x;
        const uint32_t key = key_of(ids[base + min(j, n - 1)], V);
        k[j] = j < n ? key : kNoKey;
    }
    __syncthreads();
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i0 = (int)(blockIdx.x % per_tile) * 64, i = i0 + lane;
    const uint32_t mine = k[i];
    const int from = wave * SHARE;
    int rank = 0;
    auto four = [&](int j) __attribute__((always_inline)) { return *reinterpret_cast<const u32x4 *>(k + j); };
    if (from < n) {
#pragma unroll 16
        for (int j = from; j < from + SHARE; j += 4) {
            const u32x4 q = four(j);
            if (j < i0) {  // equal keys before the 64 come first
                rank += (q[0] <= mine) + (q[1] <= mine) + (q[2] <= mine) + (q[3] <= mine);
            } else if (j >= i0 + 64) {
                rank += (q[0] < mine) + (q[1] < mine) + (q[2] < mine) + (q[3] < mine);
            } else {  // among the 64 themselves, by position
#pragma unroll
                for (int e = 0; e < 4; ++e) rank += q[e] < mine || (q[e] == mine && j - i0 + e < lane);
            }
        }
    }
    count[wave][lane] = rank;
    __syncthreads();
    if (wave == 0 && i < n) {
        rank = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) rank += count[w][lane];
        keys[base + rank] = mine;
        order[base + rank] = (int32_t)(base + i);
    }
}

// Joins up to kFan sorted lists of kTile keys: 256 keys a workgroup, which
// holds the group's keys in LDS.  A key's place is its place in its own list
// plus the keys before it in every other one (those equal to it too, in an
// earlier list): a thread counts those of a quarter of the lists, by four
// binary searches at a time.
__global__ __launch_bounds__(1024) void merge_tiles_kernel(const uint32_t *__restrict__ keys,
                                                           const int32_t *__restrict__ order,
                                                           uint32_t *__restrict__ keys_out,
                                                           int32_t *__restrict__ order_out, int64_t T) {
    extern __shared__ __attribute__((aligned(16))) uint32_t held[];
    __shared__ int count[4][256];
    static_assert(kTile == 1024 && kFan % 16 == 0, "a load of the workgroup is one list");
    const int64_t mine = blockIdx.x / (kTile / 256);             // the list of this workgroup's keys
    const int64_t first = mine / kFan * kFan;                    // the group's first list
    const int lists = (int)min((int64_t)kFan, (T - first * kTile + kTile - 1) / kTile);
    const int own = (int)(mine - first);
    for (int l = 0; l < lists; l += 4) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int64_t j = first * kTile + (l + u) * kTile + threadIdx.x;
            const uint32_t key = keys[min(j, T - 1)];
            held[(l + u) * kTile + threadIdx.x] = j < T ? key : kNoKey;
        }
    }
    const int slot = (int)(blockIdx.x % (kTile / 256)) * 256 + (threadIdx.x & 255);  // in its list
    const int quarter = threadIdx.x >> 8;
    const int64_t i = mine * kTile + slot;
    const int32_t from = order[min(i, T - 1)];
    __syncthreads();
    const uint32_t key = held[own * kTile + slot];
    int at = 0;
    for (int l = quarter * 4; l < lists; l += 16) {
        int pos[4] = {};
#pragma unroll
        for (int step = kTile / 2; step > 0; step >>= 1) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t q = held[(l + u) * kTile + pos[u] + step - 1];
                pos[u] += (l + u < own ? q <= key : q < key) ? step : 0;
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // one key is left
            const uint32_t q = held[(l + u) * kTile + pos[u]];
            pos[u] += (l + u < own ? q <= key : q < key) ? 1 : 0;
            at += l + u == own ? 0 : pos[u];
        }
    }
    count[quarter][threadIdx.x & 255] = at;
    __syncthreads();
    if (quarter == 0 && i < T) {
        at += slot + count[1][threadIdx.x] + count[2][threadIdx.x] + count[3][threadIdx.x];
        keys_out[first * kTile + at] = key;
        order_out[first * kTile + at] = from;
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

// The same for longer lists, of `len` keys each, which stay in memory.
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

// A thread's eight columns of a row of D: [at, at + 8), of which it writes those
// from the skip-th on.  A row's last vector is moved back to end with the row,
// so that the many rows that are read are read as whole vectors.  TINY: D < 8,
// one thread's columns, read one by one.
template <bool TINY>
struct Cols {
    int64_t at;
    int skip, n;
    __device__ __forceinline__ Cols(int64_t i, int64_t D) {
        at = TINY ? 0 : min(i, D - 8);
        skip = TINY ? 0 : (int)(i - at);
        n = TINY ? (int)D : 8;
    }
    template <typename T>
    __device__ __forceinline__ void load(const T *row, float (&v)[8]) const {
        if constexpr (TINY) load_n(row, n, v);
        else load8(row + at, v);
    }
    // Adds rows row(0) .. row(7), of which the first `many` count, in order;
    // all eight are read at once.
    template <typename T, typename F>
    __device__ __forceinline__ void add8(F &&row, int64_t many, float (&s)[8]) const {
        read8<T>(row, [&](int q, auto &&u) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] += q < many ? u(e) : 0.f;
        });
    }
    // use(q, value of element e) for q = 0 .. 7, after all eight rows are read.
    template <typename T, typename F, typename G>
    __device__ __forceinline__ void read8(F &&row, G &&use) const {
        if constexpr (TINY) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                float u[8];
                load_n(row(q), n, u);
                use(q, [&](int e) { return u[e]; });
            }
        } else {
            Raw8<T> u[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) u[q].load(row(q) + at);
            hold(u);
#pragma unroll
            for (int q = 0; q < 8; ++q) use(q, [&](int e) { return u[q][e]; });
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T *row, const float (&v)[8]) const {
        if (!TINY && skip == 0) {
            stream8(row + at, v);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e >= skip && e < n) row[at + e] = (T)v[e];
        }
    }
};

// A row's sum, scaled and, with `accumulate`, added to what the row holds.
template <typename WT, bool TINY>
__device__ __forceinline__ void finish_row(WT *row, const Cols<TINY> &my, const float (&sum)[8], float scale,
                                           int32_t accumulate) {
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = sum[e] * scale;
    if (accumulate) {  // (elements that it skips may be new already: they are not written)
        float u[8];
        my.load(row, u);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += u[e];
    }
    my.store(row, s);
}

// A chunk of the sorted tokens, a thread's columns: a run of equal ids that lies
// in the chunk is summed and written to its row of dW; one that comes in from
// the chunk before is summed into slot 0 of the chunk's pieces; one that begins
// here and goes on into slot 1.  The rows of eight tokens are
// in flight at a time, whatever runs they belong to.
template <typename DT, typename WT, bool TINY>
__device__ __forceinline__ void sum_chunk(const uint32_t *k, int n, uint32_t V, const int32_t *__restrict__ order,
                                          const DT *__restrict__ dX, int64_t ldx, int64_t D, const Cols<TINY> &my, float scale,
                                          int32_t accumulate, WT *__restrict__ dW, int64_t ldw,
                                          float *__restrict__ piece) {
    constexpr int U = 8;
    auto key = [&](int j) __attribute__((always_inline)) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)k[j]); };
    float s[8] = {};
    bool in = key(0) == key(1);  // the run at hand came in from the left
    for (int j0 = 0; j0 < n; j0 += U) {
        if (key(j0 + 1) >= V) return;  // padding sorts last
        bool done = false;
        my.template read8<DT>(
            [&](int q) __attribute__((always_inline)) { return dX + (int64_t)order[min(j0 + q, n - 1)] * ldx; },
            [&](int q, auto &&u) __attribute__((always_inline)) {
                const int j = j0 + q;
                done = done || j >= n || key(j + 1) >= V;
                if (done) return;
                const uint32_t v = key(j + 1);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] += u(e);
                const bool on = key(j + 2) == v;
                if (on && j + 1 < n) return;
                // the run, or this chunk's part of it, is complete
                if (in) {
                    my.store(piece, s);
                } else if (on) {
                    my.store(piece + D, s);
                } else {
                    finish_row(dW + (int64_t)v * ldw, my, s, scale, accumulate);
                }
                in = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) s[e] = 0.f;
            });
        if (done) return;
    }
}

// Workgroups [0, sums): chunk blockIdx.x / spans, and of its columns a span of
// 8 a thread.  The others, if dW is filled here: the rows without a token among
// fill.rows at a time.  Sums and fill in one launch took 431 us for 32768 tokens
// in 50257 rows of 8192, and 203 + 250 one after the other: the sums alone leave
// most of HBM's rate unused.
template <typename DT, typename WT, bool TINY>
__global__ __launch_bounds__(256) void sums_kernel(const uint32_t *__restrict__ keys, const int32_t *__restrict__ order,
                                                   int64_t T, int64_t V, int32_t chunk, int32_t sums, int32_t spans,
                                                   const DT *__restrict__ dX, int64_t ldx, int64_t D, float scale,
                                                   int32_t accumulate, WT *__restrict__ dW, int64_t ldw,
                                                   float *__restrict__ pieces, Fill fill) {
    __shared__ uint32_t k[kChunk + 2];  // the chunk's keys between their neighbours; or whether a row has no token
    if ((int)blockIdx.x < sums) {
        const int64_t c = blockIdx.x / spans, a = c * chunk;
        const int n = (int)min((int64_t)chunk, T - a);
        for (int j = threadIdx.x; j < n + 2; j += blockDim.x)
            k[j] = a + j - 1 >= 0 && a + j - 1 < T ? keys[a + j - 1] : kNoKey;
        __syncthreads();
        const int64_t i = ((int64_t)(blockIdx.x % spans) * blockDim.x + threadIdx.x) * 8;
        if (i < D)
            sum_chunk(k, n, (uint32_t)V, order + a, dX, ldx, D, Cols<TINY>(i, D), scale, accumulate, dW, ldw, pieces + 2 * c * D);
        return;
    }
    const int64_t step = (int64_t)(gridDim.x - sums) * fill.rows;
    for (int64_t v0 = (int64_t)(blockIdx.x - sums) * fill.rows; v0 < V; v0 += step) {
        if ((int)threadIdx.x < fill.rows) {
            const int64_t v = v0 + threadIdx.x, at = before<false>(keys, T, (uint32_t)min(v, V));
            k[threadIdx.x] = v < V && (at == T || keys[at] != (uint32_t)v);
        }
        __syncthreads();
        for (int r = 0; r < fill.rows; ++r)
            if (k[r]) fill_row(fill, v0 + r);
        __syncthreads();
    }
}

// Rows of dW whose run goes past the chunk it begins in (workgroup x: chunk):
// its pieces, eight in flight at a time, added in order.
template <typename WT, bool TINY>
__global__ __launch_bounds__(256) void join_kernel(const uint32_t *__restrict__ keys, int64_t T, int64_t V,
                                                   int32_t chunk, int64_t D, const float *__restrict__ pieces,
                                                   float scale, int32_t accumulate, WT *__restrict__ dW, int64_t ldw) {
    const int64_t c = blockIdx.x, a = c * chunk, b = min(a + chunk, T);
    // its last key and the one after it, the one before the chunk and its first
    const uint32_t v = keys[b - 1], next = keys[min(b, T - 1)], prev = keys[max(a - 1, (int64_t)0)], head = keys[a];
    if (v >= V || b == T || next != v) return;          // it ends here
    if (a > 0 && prev == v && head == v) return;        // it does not begin here
    // the chunks that it goes on into begin with v
    int64_t more = 0;
    for (;; more += 64) {
        const int64_t at = (c + 1 + more + (threadIdx.x & 63)) * chunk;
        const uint64_t with = __ballot(at < T && keys[min(at, T - 1)] == v);
        if (with != ~0ull) {
            more += __builtin_ctzll(~with);
            break;
        }
    }
    const int64_t i = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * 8;
    if (i >= D) return;
    const Cols<TINY> my(i, D);
    float s[8];
    my.load(pieces + (2 * c + 1) * D, s);
    for (int64_t m = 1; m <= more; m += 8)
        my.template add8<float>(
            [&](int q) __attribute__((always_inline)) { return pieces + 2 * (c + min(m + q, more)) * D; }, more - m + 1, s);
    finish_row(dW + (int64_t)v * ldw, my, s, scale, accumulate);
}

// ---- host ---------------------------------------------------------------------------

// Short lists, and short rows, take short chunks: more workgroups, each with
// fewer rows to add one after another.
constexpr int64_t kShortList = 8192, kShortRow = 512;
int32_t chunk_of(int64_t T, int64_t D) { return T <= kShortList ? 16 : D <= kShortRow ? 32 : kChunk; }
// Elements of the chunks' pieces.
int64_t pieces_of(int64_t T, int64_t D) { return ceil_div(T, chunk_of(T, D)) * 2 * D; }
int64_t up4(int64_t x) { return (x + 3) / 4 * 4; }
// Threads of a workgroup that sums rows of D elements, and workgroups a row.
int64_t threads_of(int64_t D) { return D > 1024 ? 256 : D > 512 ? 128 : 64; }
int64_t spans_of(int64_t D) { return ceil_div(D, threads_of(D) * 8); }

// The workspace of a gradient: two sets of keys and positions (the sort goes
// from one to the other), the pieces.
struct Work {
    uint64_t keys[2], order[2], pieces, bytes;
};
Work work_of(int64_t T, int64_t D) {
    Work w;
    uint64_t at = 0;
    for (int k = 0; k < 2; ++k) {
        w.keys[k] = at;
        at += up256((uint64_t)T * 4);
        w.order[k] = at;
        at += up256((uint64_t)T * 4);
    }
    w.pieces = at;
    // Where the chunks get longer, so where their pieces get fewer, the room
    // stays: a workspace for T tokens of D columns holds any fewer of both.
    const int64_t t = min64(T, kShortList), d = min64(D, kShortRow);
    const uint64_t most = max64(pieces_of(T, D), max64(pieces_of(t, D), pieces_of(T, d)));
    at += up256(most * 4);
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
        if (p->D < 8)
            hipLaunchKernelGGL((embed_fwd_kernel<WT, XT, 16, true>), dim3((unsigned)min64(ceil_div(p->T, 16), kMostGroups)),
                               dim3(256), 0, s, ids, wide, p->T, p->V, p->D, static_cast<const WT *>(W), ldw, p->scale,
                               static_cast<XT *>(X), ldx);
        else
            hipLaunchKernelGGL((embed_fwd_kernel<WT, XT, L, false>), g, dim3(256), 0, s, ids, wide, p->T, p->V, p->D,
                               static_cast<const WT *>(W), ldw, p->scale, static_cast<XT *>(X), ldx);
        return hipGetLastError();
    };
    if (vecs <= 16) return go(std::integral_constant<int, 16>{});
    if (vecs <= 64) return go(std::integral_constant<int, 64>{});
    return go(std::integral_constant<int, 256>{});
}

template <typename DT, typename WT, bool TINY>
hipError_t run_bwd(const zi_embedding *p, const void *ids, const void *dX, void *dW, char *work, hipStream_t s) {
    const int64_t T = p->T, V = p->V, D = p->D;
    const int64_t ldw = p->ldw ? p->ldw : D, ldx = p->ldx ? p->ldx : D;
    const int32_t chunk = chunk_of(T, D);
    const Work w = work_of(T, D);
    uint32_t *keys[2] = {};
    int32_t *order[2] = {};
    float *pieces = nullptr;
    int k = 0;
    hipError_t e;
    // Zeros.  Where most rows stay without a token, all of dW is filled beside the
    // sort, which leaves the device nearly idle; else the rows without a token
    // beside the sums, which writes no row twice.  A workgroup looks at as many
    // rows as 64 KiB hold (1 MiB: 3 % slower), fewer if there would be too few workgroups.
    Fill fill{};
    fill.base = reinterpret_cast<char *>(dW);
    fill.V = V;
    fill.stride = ldw * (int64_t)sizeof(WT);
    fill.bytes = D * (int64_t)sizeof(WT);
    fill.rows = (int32_t)max64(1, min64(min64((1 << 16) / fill.bytes, V / 1024), kMostRows));
    const int64_t fills = p->accumulate ? 0 : min64(ceil_div(V, fill.rows), kMostGroups);
    const bool at_sort = T > 0 && T <= V / 8;
    if (T > 0) {
        for (int j = 0; j < 2; ++j) {
            keys[j] = reinterpret_cast<uint32_t *>(work + w.keys[j]);
            order[j] = reinterpret_cast<int32_t *>(work + w.order[j]);
        }
        pieces = reinterpret_cast<float *>(work + w.pieces);
        const int64_t lists = T <= kOneTile ? 1 : ceil_div(T, kTile);
        const int32_t per_tile = (int32_t)(lists > 1 ? kTile / 64 : ceil_div(T, 64));
        const int32_t sorts = (int32_t)lists * per_tile;
        const dim3 g((unsigned)(sorts + (at_sort ? fills : 0)));
        auto sort = [&](auto tile) {
            constexpr int TILE = decltype(tile)::value;
            if (p->ids64)
                hipLaunchKernelGGL((sort_tile_kernel<TILE, int64_t>), g, dim3(1024), 0, s, static_cast<const int64_t *>(ids),
                                   T, V, keys[0], order[0], sorts, per_tile, fill);
            else
                hipLaunchKernelGGL((sort_tile_kernel<TILE, int32_t>), g, dim3(1024), 0, s, static_cast<const int32_t *>(ids),
                                   T, V, keys[0], order[0], sorts, per_tile, fill);
            return hipGetLastError();
        };
        e = T > kTile && lists == 1 ? sort(std::integral_constant<int, kOneTile>{}) : sort(std::integral_constant<int, kTile>{});
        if (e != hipSuccess) return e;
        if (lists > 1) {
            hipLaunchKernelGGL(merge_tiles_kernel, dim3((unsigned)lists * (kTile / 256)), dim3(1024),
                               (unsigned)(min64(up4(lists), kFan) * kTile * 4), s, keys[0], order[0], keys[1], order[1], T);
            if ((e = hipGetLastError()) != hipSuccess) return e;
            k = 1;
            for (int64_t len = (int64_t)kTile * kFan; len < T; len *= kFan, k ^= 1) {
                hipLaunchKernelGGL(merge_kernel, dim3((unsigned)ceil_div(T, 256)), dim3(256), 0, s, keys[k], order[k],
                                   keys[k ^ 1], order[k ^ 1], T, len);
                if ((e = hipGetLastError()) != hipSuccess) return e;
            }
        }
    }
    const int64_t threads = threads_of(D), chunks = ceil_div(T, chunk), spans = spans_of(D);
    const int64_t sums = chunks * spans, groups = sums + (at_sort ? 0 : fills);
    if (groups == 0) return hipSuccess;
    hipLaunchKernelGGL((sums_kernel<DT, WT, TINY>), dim3((unsigned)groups), dim3((unsigned)threads), 0, s, keys[k], order[k], T, V,
                       chunk, (int32_t)sums, (int32_t)spans, static_cast<const DT *>(dX), ldx, D, p->scale, p->accumulate,
                       static_cast<WT *>(dW), ldw, pieces, fill);
    if ((e = hipGetLastError()) != hipSuccess || chunks < 2) return e;
    hipLaunchKernelGGL((join_kernel<WT, TINY>), dim3((unsigned)chunks, (unsigned)spans), dim3((unsigned)threads), 0, s, keys[k], T,
                       V, chunk, D, pieces, p->scale, p->accumulate, static_cast<WT *>(dW), ldw);
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
    // the sort takes sixteen threads a token, and a launch's threads are a 32-bit number
    if (p->T < 0 || p->T > (1 << 27)) return fail(ZI_ERR_SHAPE, "T = %lld: 0 .. 2^27 tokens", (long long)p->T);
    if (p->V < 1 || p->V > INT32_MAX) return fail(ZI_ERR_SHAPE, "V = %lld: 1 .. 2^31 - 1 rows", (long long)p->V);
    // spans of columns are a grid's second dimension
    if (p->D < 1 || p->D > 65535 * (int64_t)2048) return fail(ZI_ERR_SHAPE, "D = %lld is out of range", (long long)p->D);
    // so do the sums'
    if (ceil_div(p->T, chunk_of(p->T, p->D)) * spans_of(p->D) * threads_of(p->D) > (int64_t)UINT32_MAX - kMostGroups * 256)
        return fail(ZI_ERR_SHAPE, "T = %lld rows of D = %lld are too many", (long long)p->T, (long long)p->D);
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
    return work_of(T, D).bytes;
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
        char *work = static_cast<char *>(workspace);
        return p->D < 8 ? run_bwd<decltype(x), decltype(w), true>(p, ids, dX, dW, work, s)
                        : run_bwd<decltype(x), decltype(w), false>(p, ids, dX, dW, work, s);
    });
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "embedding gradient: %s", hipGetErrorString(e));
    return ZI_OK;
}
