// zi_route.hip -- the router of a mixture of experts and the sum of its experts' rows.
//
// Router, forward: for every token the k experts with the largest logits, their
// softmax weights, and the (token, choice) pairs sorted by expert.  The work is a
// few instructions a logit, so what counts is that the selection takes few
// of them and that there are few launches:
//   choose  L lanes share a token (8 for up to 128 experts, 64 for 1024), so a
//           wave takes 64 / L tokens side by side.  Logits are compared as ordered
//           integers, in which 0 stands for an expert that cannot be chosen.
//   place   a stable counting sort.  A token has an expert once, so the rank of a
//           pair among its expert's is a count of tokens: a bit mask of 128 tokens
//           for every expert, whose bits are set in any order and counted below
//           the token.  What the blocks before hold is summed by every block for
//           itself (at most kMostBlocks counts an expert), which takes less than a
//           third launch.
// Up to kOneTokens tokens both run in one workgroup and one launch.  (32768 tokens of 256
// fp32 logits, k = 8: choose 12.4 us, 2.7 TB/s of logits, bound by its instructions;
// place 7.3, bound by its launch and the chain from counts to masks to places.  One
// token of 64: 6.9 us, the call.)
//
// Backward: dl = p (g - sum p g), g the weights' gradients at the chosen experts, lanes
// as in choose, everything in registers.  (32768 tokens of 128 bf16, k = 6: 8.4 us,
// 2.1 TB/s, bound by instructions.)
//
// Combination: Y_t = sum_j w_tj Z[slot_tj], and backward dZ[slot_tj] = w_tj dY_t,
// dw_tj = dY_t . Z[slot_tj].  Both are bound by HBM: every row is read or written
// once, whole vectors of eight elements, written past the caches.  (Forward, 32768 tokens
// of 4 x 8192 bf16: 507 us, 5.2 TB/s.  Backward, 4099 of 6 x 5003 fp16: 130 us, 4.1 TB/s.)
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "zi_host.h"
#include "zi_vec.h"

namespace zi {
namespace {

constexpr int kOneThreads = 256, kThreads = 1024;  // of a workgroup that does everything; of the others
constexpr int kMostChoices = 32;
constexpr int kMaskTokens = 128;          // tokens of a mask: four words an expert
constexpr int kMostBlocks = 512;
constexpr int kOneTokens = 64;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- maxima and sums over L lanes ------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
}
// Over L consecutive lanes (8 .. 64, a power of two); every lane gets the result.
// Up to 16 lanes by DPP: the other of a pair, the other pair of four, the mirrored
// half of eight, the mirrored half of sixteen.
template <int L, typename F>
__device__ __forceinline__ uint32_t lanes(uint32_t x, F &&f) {
    x = f(x, dpp<0xb1>(x));
    x = f(x, dpp<0x4e>(x));
    x = f(x, dpp<0x141>(x));
    if constexpr (L >= 16) x = f(x, dpp<0x140>(x));
    if constexpr (L >= 32) x = f(x, (uint32_t)__shfl_xor((int)x, 16, 64));
    if constexpr (L >= 64) x = f(x, (uint32_t)__shfl_xor((int)x, 32, 64));
    return x;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
    return lanes<L>(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
    return __builtin_bit_cast(float, lanes<L>(__builtin_bit_cast(uint32_t, x), [](uint32_t a, uint32_t b) {
                                  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
                              }));
}

// A logit as an integer of the same order; 0: -inf or NaN, which are not chosen.
// (-0 counts as 0.)
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);
    const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return x > -INFINITY ? k : 0u;
}
__device__ __forceinline__ float logit_of(uint32_t k) {
    return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// e^x of x <= 0 for a sum that has a one in it: 2^(x log2 e), the product's rounding and
// log2 e's own put back to first order, so that the error is an ulp or so of the
// instruction's.  Below 2^-126 zero, and NaN is not kept.  (Six instructions for some 15 of
// expf; of the choice among 22251 x 311 logits it takes 4 us off 20.)
__device__ __forceinline__ float exp_below(float x) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596299e-8f;  // log2 e
    x = fmaxf(x, -104.f);
    const float y = x * kHi, rest = __builtin_fmaf(x, kLo, __builtin_fmaf(x, kHi, -y));
    const float e = __builtin_amdgcn_exp2f(y);
    return __builtin_fmaf(e, rest * 0.693147181f, e);
}

// The V logits of a lane's experts, -inf past the last one (n of them are left).
template <int V, typename LT>
__device__ __forceinline__ void load_logits(const LT *p, int n, float (&x)[V]) {
#pragma unroll
    for (int c = 0; c < V; c += 8) {
        float v[8];
        load_n(p + c, n - c, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[c + e] = c + e < n ? v[e] : -INFINITY;
    }
}

// ---- choice ------------------------------------------------------------------------------

// Of each group of L lanes, which are of one wave: its lanes' maxima, how many
// candidates it has, and those; then its choices.
struct Pick {
    uint32_t lo, hi;  // a candidate: ~index, key (one number, of its order); a choice: index, logit
};
template <int GROUPS, int L>
struct Chosen {
    uint32_t most[GROUPS][L];
    uint32_t count[GROUPS];
    __attribute__((aligned(16))) Pick pick[GROUPS][kMostChoices];
};
// The lanes of a wave access LDS in order; this keeps the compiler to it.
__device__ __forceinline__ void lds_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// The choices of tokens [t0, t1), counted in hist (shared, E counts).
//
// Of the lanes' maxima the k-th largest is a bound that at least k logits reach.  Those
// that do, some 12 of 256 for k = 8, are gathered in LDS and ranked by counting, all
// lanes at once.  Where there are more than kMostChoices (many equal logits), or k is
// more than there are lanes, the choices are found one after another.  (32768 tokens,
// 256 experts, k = 8: 19.7 us one after another, bound by instructions.)
template <int THREADS, typename LT, int L, int V>
__device__ __forceinline__ void choose(const LT *logits, int64_t ldl, int64_t t0, int64_t t1, int E, int k, int normalize,
                                       int32_t *ids, float *weights, uint32_t *hist, Chosen<THREADS / L, L> &lds) {
    const int lane = threadIdx.x & (L - 1), group = threadIdx.x / L;
    const int first = lane * V;  // this lane's first expert
    const int shift = (threadIdx.x & 63) & ~(L - 1);
    Pick *pick = lds.pick[group];
    for (int64_t base = t0; base < t1; base += THREADS / L) {
        const int64_t t = base + group;
        const int n = t < t1 ? E - first : 0;
        float x[V];
        load_logits<V>(logits + (t < t1 ? t : t0) * ldl + first, n, x);
        uint32_t key[V], bad = 0, most = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            key[v] = key_of(x[v]);
            bad |= x[v] != x[v] ? 1u : 0u;
            most = key[v] > most ? key[v] : most;
        }
        int found = 0;
        bool slow = k > L;
        if (!slow) {
            constexpr int PER = kMostChoices > L ? kMostChoices / L : 1;
            lds.most[group][lane] = most;
            if (lane == 0) lds.count[group] = 0;
#pragma unroll
            for (int q = 0; q < PER; ++q)
                if (lane + q * L < kMostChoices) pick[lane + q * L] = Pick{0, 0};
            lds_order();
            uint32_t above = 0;  // lanes with a larger maximum
#pragma unroll
            for (int i = 0; i < L; ++i) above += lds.most[group][i] > most ? 1u : 0u;
            const uint32_t least = lanes<L>(above < (uint32_t)k ? most : ~0u, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
            const uint32_t bound = least > 1u ? least : 1u;
            uint32_t mine = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) mine += key[v] >= bound ? 1u : 0u;
            uint32_t at = mine ? atomicAdd(&lds.count[group], mine) : 0u;
            lds_order();
            const uint32_t all = lds.count[group];
            slow = __ballot(all > (uint32_t)kMostChoices) != 0;
            if (!slow) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (key[v] >= bound) pick[at++] = Pick{~(uint32_t)(first + v), key[v]};
                lds_order();
                uint64_t own[PER];
                uint32_t rank[PER] = {};
#pragma unroll
                for (int q = 0; q < PER; ++q) {
                    const Pick p = pick[(lane + q * L) & (kMostChoices - 1)];
                    own[q] = (uint64_t)p.hi << 32 | p.lo;
                }
                // (entries past the last are zeros, which no candidate is below)
                for (uint32_t j = 0; __ballot(j < all) != 0; j += 2) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const Pick p = pick[j + h];
                        const uint64_t other = (uint64_t)p.hi << 32 | p.lo;
#pragma unroll
                        for (int q = 0; q < PER; ++q) rank[q] += other > own[q] ? 1u : 0u;
                    }
                }
                lds_order();
#pragma unroll
                for (int q = 0; q < PER; ++q)
                    if (own[q] && rank[q] < (uint32_t)k && lane + q * L < kMostChoices)
                        pick[rank[q]] = Pick{~(uint32_t)own[q], __builtin_bit_cast(uint32_t, logit_of((uint32_t)(own[q] >> 32)))};
                found = (int)(all < (uint32_t)k ? all : (uint32_t)k);
            }
        }
        if (slow) {
            for (int j = 0; j < k; ++j) {
                uint32_t m = key[0];
#pragma unroll
                for (int v = 1; v < V; ++v) m = key[v] > m ? key[v] : m;
                const uint32_t best = lanes_max<L>(m);
                const uint64_t having = __ballot(m == best) >> shift;
                if (__ballot(best != 0) == 0) break;  // no token of the wave has another expert
                if (best == 0) continue;
                ++found;
                // the lowest lane that has it gives it up, its first one
                const bool wins = lane == __builtin_ctzll(having);
                bool still = wins;
                int at = 0;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const bool hit = still & (key[v] == best);
                    still = still & !hit;
                    key[v] = hit ? 0u : key[v];
                    at = hit ? v : at;
                }
                if (wins) pick[j] = Pick{(uint32_t)(first + at), __builtin_bit_cast(uint32_t, logit_of(best))};
            }
        }
        lds_order();
        const float top = found ? __builtin_bit_cast(float, pick[0].hi) : 0.f;
        float total = 0.f;
        if (normalize) {
            for (int j = lane; j < found; j += L) total += expf(__builtin_bit_cast(float, pick[j].hi) - top);
        } else {  // over all experts
#pragma unroll
            for (int v = 0; v < V; ++v) total += exp_below(x[v] - top);
        }
        total = lanes_sum<L>(total);
        if (lanes_max<L>(bad) || top == INFINITY) total = NAN;
        if (t < t1) {
            for (int j = lane; j < k; j += L) {
                const bool is = j < found;
                const int id = is ? (int)pick[j].lo : -1;
                ids[t * k + j] = id;
                weights[t * k + j] = is ? expf(__builtin_bit_cast(float, pick[j].hi) - top) / total : 0.f;
                if (is) atomicAdd(hist + id, 1u);
            }
        }
        lds_order();
    }
}

// Counts a row holds: a whole number of words of bytes.
__host__ __device__ constexpr int row_of(int E) { return (E + 3) / 4 * 4; }

// ---- placement ---------------------------------------------------------------------------

// base[e] = before[e] + the sum of all[] of the experts before e; returns the sum
// of all of them.  THREADS threads, at most 1024 experts; part: a word a wave.
template <int THREADS>
__device__ __forceinline__ uint32_t bases_of(const uint32_t *all, const uint32_t *before, int E, uint32_t *base,
                                             int32_t *offsets, uint32_t *part) {
    constexpr int Q = 1024 / THREADS;
    const int first = threadIdx.x * Q, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t mine[Q], sum = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        mine[q] = first + q < E ? all[first + q] : 0u;
        sum += mine[q];
    }
    uint32_t scan = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t y = (uint32_t)__shfl_up((int)scan, d, 64);
        scan += lane >= d ? y : 0u;
    }
    if (lane == 63) part[wave] = scan;
    __syncthreads();
    uint32_t at = scan - sum, total = 0;
    for (int w = 0; w < THREADS / 64; ++w) {
        at += w < wave ? part[w] : 0u;
        total += part[w];
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        if (first + q < E) {
            base[first + q] = at + (before ? before[first + q] : 0u);
            if (offsets) offsets[first + q] = (int32_t)at;
        }
        at += mine[q];
    }
    if (offsets && threadIdx.x == 0) offsets[E] = (int32_t)total;
    __syncthreads();
    return total;
}

// rows and slots of tokens [t0, t1); base: the next place of each expert; mask: 4 E words.
template <int THREADS>
__device__ __forceinline__ void place(const int32_t *ids, int64_t t0, int64_t t1, int E, int k, uint32_t *base,
                                      uint32_t *mask, int32_t *rows, int32_t *slots) {
    for (int64_t s0 = t0; s0 < t1; s0 += kMaskTokens) {
        const int n = (int)(t1 - s0 < kMaskTokens ? t1 - s0 : kMaskTokens) * k;
        for (int i = threadIdx.x; i < 4 * E; i += THREADS) mask[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += THREADS) {
            const int e = ids[s0 * k + i];
            const uint32_t t = (uint32_t)i / (uint32_t)k;
            if (e >= 0) atomicOr(mask + 4 * e + (t >> 5), 1u << (t & 31));
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += THREADS) {
            const int e = ids[s0 * k + i];
            const uint32_t t = (uint32_t)i / (uint32_t)k;
            int32_t slot = -1;
            if (e >= 0) {
                uint32_t rank = __builtin_popcount(mask[4 * e + (t >> 5)] & ((1u << (t & 31)) - 1u));
                for (uint32_t w = 0; w < (t >> 5); ++w) rank += __builtin_popcount(mask[4 * e + w]);
                slot = (int32_t)(base[e] + rank);
                rows[slot] = (int32_t)(s0 + t);
            }
            slots[s0 * k + i] = slot;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += THREADS) {
            uint32_t c = 0;
#pragma unroll
            for (int w = 0; w < 4; ++w) c += __builtin_popcount(mask[4 * e + w]);
            base[e] += c;
        }
        __syncthreads();
    }
}

// Everything in one workgroup.
template <typename LT, int L, int V>
__global__ __launch_bounds__(kOneThreads) void route_kernel(const LT *logits, int64_t ldl, int T, int E, int k, int normalize,
                                                               int32_t *ids, float *weights, int32_t *offsets, int32_t *rows,
                                                               int32_t *slots) {
    __shared__ Chosen<kOneThreads / L, L> out;
    __shared__ uint32_t hist[L * V], base[L * V], mask[4 * L * V], part[kOneThreads / 64];
    for (int e = threadIdx.x; e < E; e += kOneThreads) hist[e] = 0;
    __syncthreads();
    choose<kOneThreads, LT, L, V>(logits, ldl, 0, T, E, k, normalize, ids, weights, hist, out);
    __threadfence_block();  // the ids are read again
    __syncthreads();
    const int total = (int)bases_of<kOneThreads>(hist, nullptr, E, base, offsets, part);
    place<kOneThreads>(ids, 0, T, E, k, base, mask, rows, slots);
    for (int i = total + threadIdx.x; i < T * k; i += kOneThreads) rows[i] = -1;
}

// Block b: tokens [b step, (b + 1) step), its counts in row b of counts: bytes where a
// block has at most 128 tokens (every other block reads them: 256 blocks and experts in 32 bits
// took 10.3 us, most of it for the 64 MB).
template <typename LT, int L, int V>
__global__ __launch_bounds__(kThreads) void choose_kernel(const LT *logits, int64_t ldl, int64_t T, int64_t step, int E,
                                                                int k, int normalize, int32_t *ids, float *weights,
                                                                void *counts) {
    __shared__ Chosen<kThreads / L, L> out;
    __shared__ uint32_t hist[L * V];
    for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
    __syncthreads();
    const int64_t t0 = blockIdx.x * step, t1 = t0 + step < T ? t0 + step : T;
    choose<kThreads, LT, L, V>(logits, ldl, t0, t1, E, k, normalize, ids, weights, hist, out);
    __syncthreads();
    const int64_t row = (int64_t)blockIdx.x * row_of(E);
    for (int e = threadIdx.x; e < row_of(E); e += kThreads) {
        const uint32_t n = e < E ? hist[e] : 0;
        if (step <= kMaskTokens) static_cast<uint8_t *>(counts)[row + e] = (uint8_t)n;
        else static_cast<uint32_t *>(counts)[row + e] = n;
    }
}

__global__ __launch_bounds__(kThreads) void place_kernel(const int32_t *ids, int64_t T, int64_t step, int E, int k,
                                                              const void *counts, int32_t *offsets, int32_t *rows,
                                                              int32_t *slots) {
    __shared__ uint32_t all[1024], before[1024], base[1024], mask[4 * 1024], part[kThreads / 64];
    const int b = blockIdx.x, blocks = gridDim.x;
    for (int e = threadIdx.x; e < E; e += kThreads) all[e] = before[e] = 0;
    __syncthreads();
    // four experts a thread; the threads left over share the blocks
    const int words = row_of(E) / 4, shares = kThreads / words, share = threadIdx.x / words, w = threadIdx.x - share * words;
    if (share < shares) {
        uint32_t sum[4] = {}, low[4] = {};
        if (step <= kMaskTokens) {
            // sums of two bytes a word: a share has at most 128 of the 512 blocks (256 words
            // at most), so they stay below 2^16
            static_assert(kMostBlocks / (kThreads / (ZI_ROUTE_EXPERTS / 4)) * kMaskTokens < 65536, "16-bit sums");
            uint32_t s0 = 0, s1 = 0, l0 = 0, l1 = 0;
            const uint32_t *row = static_cast<const uint32_t *>(counts) + w;
#pragma unroll 8
            for (int c = share; c < blocks; c += shares) {
                const uint32_t n = row[(int64_t)c * words], n0 = n & 0x00ff00ffu, n1 = (n >> 8) & 0x00ff00ffu;
                s0 += n0;
                s1 += n1;
                l0 += c < b ? n0 : 0u;
                l1 += c < b ? n1 : 0u;
            }
            sum[0] = s0 & 0xffffu, sum[1] = s1 & 0xffffu, sum[2] = s0 >> 16, sum[3] = s1 >> 16;
            low[0] = l0 & 0xffffu, low[1] = l1 & 0xffffu, low[2] = l0 >> 16, low[3] = l1 >> 16;
        } else {
            const u32x4_u *row = static_cast<const u32x4_u *>(counts) + w;
#pragma unroll 4
            for (int c = share; c < blocks; c += shares) {
                const u32x4_u n = row[(int64_t)c * words];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    sum[q] += n[q];
                    low[q] += c < b ? n[q] : 0u;
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (4 * w + q < E) {
                atomicAdd(all + 4 * w + q, sum[q]);
                atomicAdd(before + 4 * w + q, low[q]);
            }
        }
    }
    __syncthreads();
    const int64_t total = bases_of<kThreads>(all, before, E, base, b == 0 ? offsets : nullptr, part);
    const int64_t t0 = b * step, t1 = t0 + step < T ? t0 + step : T;
    place<kThreads>(ids, t0, t1, E, k, base, mask, rows, slots);
    for (int64_t i = total + (int64_t)b * kThreads + threadIdx.x; i < T * k; i += (int64_t)blocks * kThreads) rows[i] = -1;
}

// ---- backward ----------------------------------------------------------------------------

template <typename LT, int L, int V, bool NORM>
__global__ __launch_bounds__(256) void route_bwd_kernel(const LT *logits, int64_t ldl, int64_t T, int E, int k, const int32_t *ids,
                                                        const float *weights, const float *dweights, LT *dlogits, int64_t ldd) {
    const int lane = threadIdx.x & (L - 1), first = lane * V;
    for (int64_t t = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L; t < T; t += (int64_t)gridDim.x * (256 / L)) {
        const int n = E - first;
        float p[V], g[V] = {};
        float scale = 1.f;
        if constexpr (NORM) {
#pragma unroll
            for (int v = 0; v < V; ++v) p[v] = 0.f;
        } else {
            load_logits<V>(logits + t * ldl + first, n, p);
            // the largest by its order, in which a NaN is the lowest: the sum then carries it
            uint32_t m = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) m = max(m, key_of(p[v]));
            m = lanes_max<L>(m);
            const float top = m ? logit_of(m) : 0.f;
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                p[v] = v < n ? expf(p[v] - top) : 0.f;
                sum += p[v];
            }
            sum = lanes_sum<L>(sum);
            scale = sum == 0.f ? 0.f : 1.f / sum;
        }
        float along = 0.f;
        for (int j0 = 0; j0 < k; j0 += 8) {
            int id[8];
            float d[8], w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool is = j0 + j < k;
                id[j] = is ? ids[t * k + j0 + j] : -1;
                d[j] = is ? dweights[t * k + j0 + j] : 0.f;
                w[j] = NORM && is ? weights[t * k + j0 + j] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (id[j] < 0) continue;
                if constexpr (NORM) along += w[j] * d[j];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const bool hit = id[j] == first + v;
                    g[v] += hit ? d[j] : 0.f;
                    if constexpr (NORM) p[v] = hit ? w[j] : p[v];
                }
            }
        }
        if constexpr (!NORM) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                p[v] *= scale;
                along += p[v] * g[v];
            }
            along = lanes_sum<L>(along);
        }
#pragma unroll
        for (int c = 0; c < V; c += 8) {
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = p[c + e] * (g[c + e] - along);
            store_n(dlogits + t * ldd + first + c, n - c, o);
        }
    }
}

// ---- combination -------------------------------------------------------------------------

// A row's vectors of eight elements belong to `lanes` threads in turn.  The last
// vector is moved back to end with the row; `from` is the first of its elements that
// no other vector holds.
struct Vec {
    int64_t at;
    int from;
};
__device__ __forceinline__ Vec vec_of(int64_t v, int64_t D) {
    const int64_t at = v * 8;
    return at + 8 <= D ? Vec{at, 0} : Vec{D - 8, (int)(at + 8 - D)};
}

// rows of fewer than eight elements
template <typename ZT>
__device__ __forceinline__ void load_row(const ZT *p, int64_t D, int64_t at, float (&v)[8]) {
    if (D >= 8) load8(p + at, v);
    else load_n(p, D, v);
}
template <typename ZT>
__device__ __forceinline__ void store_row(ZT *p, int64_t D, int64_t at, const float (&v)[8]) {
    if (D >= 8) stream8(p + at, v);
    else store_n(p, D, v);
}

// Rows of Z read at a time.
constexpr int kRowsAhead = 4;

template <typename ZT>
__global__ __launch_bounds__(256) void combine_fwd_kernel(const ZT *Z, int64_t ldz, int64_t R, const int32_t *slots,
                                                          const float *weights, int64_t T, int64_t D, int k, int row_threads,
                                                          ZT *Y, int64_t ldy) {
    const int per = 256 / row_threads, lane = threadIdx.x % row_threads;
    const int64_t vecs = (D + 7) / 8;
    for (int64_t t = (int64_t)blockIdx.x * per + threadIdx.x / row_threads; t < T; t += (int64_t)gridDim.x * per) {
        for (int64_t v = lane + (int64_t)blockIdx.y * row_threads; v < vecs; v += (int64_t)gridDim.y * row_threads) {
            const Vec at = D >= 8 ? vec_of(v, D) : Vec{0, 0};
            float y[8] = {};
            for (int j0 = 0; j0 < k; j0 += kRowsAhead) {
                float z[kRowsAhead][8], w[kRowsAhead];
#pragma unroll
                for (int j = 0; j < kRowsAhead; ++j) {
                    const int slot = j0 + j < k ? slots[t * k + j0 + j] : -1;
                    w[j] = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[j][e] = 0.f;
                    if (slot >= 0 && slot < R) {
                        w[j] = weights[t * k + j0 + j];
                        load_row(Z + slot * ldz, D, at.at, z[j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < kRowsAhead; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] += w[j] * z[j][e];
            }
            store_row(Y + t * ldy, D, at.at, y);
        }
    }
}

// KP rows of Z at a time, dY's vectors again from the caches for each pair: with rows
// read and written side by side memory does worse (4099 tokens of 6 x 5003 fp16: 133 us
// with two rows, 152 with four, 162 with eight; one barrier a token in place of two a
// pair, which keep the four waves on the same rows, 146).
constexpr int KP = 2;
template <typename ZT>
__global__ __launch_bounds__(256) void combine_bwd_kernel(const ZT *dY, int64_t ldy, const ZT *Z, int64_t ldz, int64_t R,
                                                          const int32_t *slots, const float *weights, int64_t T, int64_t D, int k,
                                                          int row_threads, ZT *dZ, int64_t lddz, float *dweights) {
    __shared__ float part[4][KP];
    const int per = 256 / row_threads, lane = threadIdx.x % row_threads, wave = threadIdx.x >> 6;
    const int64_t vecs = (D + 7) / 8;
    // every thread takes as many turns, since they meet
    for (int64_t t0 = (int64_t)blockIdx.x * per; t0 < T; t0 += (int64_t)gridDim.x * per) {
        const int64_t t = t0 + threadIdx.x / row_threads;
        for (int j0 = blockIdx.y * KP; j0 < k; j0 += gridDim.y * KP) {
            int64_t slot[KP];
            float w[KP], sum[KP];
#pragma unroll
            for (int j = 0; j < KP; ++j) {
                slot[j] = t < T && j0 + j < k ? slots[t * k + j0 + j] : -1;
                if (slot[j] >= R) slot[j] = -1;
                w[j] = slot[j] >= 0 ? weights[t * k + j0 + j] : 0.f;
                sum[j] = 0.f;
            }
            if (t < T) {
                for (int64_t v = lane; v < vecs; v += row_threads) {
                    const Vec at = D >= 8 ? vec_of(v, D) : Vec{0, 0};
                    float d[8];
                    Raw8<ZT> z[KP];
                    load_row(dY + t * ldy, D, at.at, d);
                    if (D >= 8) {
#pragma unroll
                        for (int j = 0; j < KP; ++j)
                            if (slot[j] >= 0) z[j].load(Z + slot[j] * ldz + at.at);
                    }
#pragma unroll
                    for (int j = 0; j < KP; ++j) {
                        if (slot[j] < 0) continue;
                        float zf[8], o[8];
                        if (D >= 8) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) zf[e] = z[j][e];
                        } else {
                            load_n(Z + slot[j] * ldz, D, zf);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            sum[j] += e >= at.from ? d[e] * zf[e] : 0.f;
                            o[e] = w[j] * d[e];
                        }
                        store_row(dZ + slot[j] * lddz, D, at.at, o);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < KP; ++j) {
                for (int m = 1; m < row_threads && m < 64; m <<= 1) sum[j] += __shfl_xor(sum[j], m, 64);
            }
            if (row_threads > 64) {
                __syncthreads();  // the sums before have been read
#pragma unroll
                for (int j = 0; j < KP; ++j)
                    if ((threadIdx.x & 63) == 0) part[wave][j] = sum[j];
                __syncthreads();
                const int waves = row_threads / 64, first = wave / waves * waves;
#pragma unroll
                for (int j = 0; j < KP; ++j) {
                    sum[j] = 0.f;
                    for (int q = 0; q < waves; ++q) sum[j] += part[first + q][j];
                }
            }
            if (lane == 0 && t < T) {
#pragma unroll
                for (int j = 0; j < KP; ++j)
                    if (j0 + j < k) dweights[t * k + j0 + j] = sum[j];
            }
        }
    }
}

// Workgroups below which a combination of few tokens is shared out further.  (31 tokens
// of 4 x 13011 bf16, backward: 22.9 us with one workgroup a token.)
constexpr int64_t kFewTokens = 512;

// ---- launches ----------------------------------------------------------------------------

// Lanes a token: the fewest with at most 8 (16) logits each.
template <typename F>
hipError_t with_lanes(int E, F &&f) {
    using std::integral_constant;
    if (E <= 64) return f(integral_constant<int, 8>{}, integral_constant<int, 8>{});
    if (E <= 128) return f(integral_constant<int, 8>{}, integral_constant<int, 16>{});
    if (E <= 256) return f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    if (E <= 512) return f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
    return f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}
template <typename F>
hipError_t with_type(int32_t d, F &&f) {
    if (d == ZI_F32) return f(float{});
    if (d == ZI_F16) return f(f16_t{});
    return f(bf16_t{});
}

// Tokens a block: at most 128, if kMostBlocks blocks then suffice, so that a SIMD's waves
// take the fewest turns with L lanes a token; of equal ones the fewest blocks, which are
// counted by each other.  (22251 tokens of 311 experts, k = 1: 24.0 us, choice and places;
// 28 with 128 tokens a block, 32 with 64.)
int64_t step_of(int64_t T, int L) {
    int64_t best = kMaskTokens * ceil_div(T, (int64_t)kMaskTokens * kMostBlocks), least = INT64_MAX;
    if (best > kMaskTokens) return best;
    for (int64_t step = kMaskTokens; step >= 32 && ceil_div(T, step) <= kMostBlocks; step -= 32) {
        const int64_t turns = ceil_div(ceil_div(T, step), 256) * ceil_div(step * L, 256);
        if (turns < least) best = step, least = turns;
    }
    return best;
}

bool known(int32_t d) { return d == ZI_F16 || d == ZI_BF16 || d == ZI_F32; }
bool aligned(const void *p, uint64_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
uint64_t size_of(int32_t d) { return d == ZI_F32 ? 4 : 2; }

zi_status check(const zi_route *r) {
    if (!r) return fail(ZI_ERR_ARG, "route is NULL");
    if (r->E < 1 || r->E > ZI_ROUTE_EXPERTS) return fail(ZI_ERR_SHAPE, "E = %d: 1 .. %d experts", r->E, ZI_ROUTE_EXPERTS);
    if (r->k < 1 || r->k > kMostChoices || r->k > r->E)
        return fail(ZI_ERR_SHAPE, "k = %d: 1 .. %d, and at most E = %d", r->k, kMostChoices, r->E);
    if (r->T < 0 || r->T > ((int64_t)1 << 30) / r->k) return fail(ZI_ERR_SHAPE, "T = %lld: T k at most 2^30", (long long)r->T);
    if ((r->ldl != 0 && r->ldl < r->E) || (r->ldd != 0 && r->ldd < r->E)) return fail(ZI_ERR_SHAPE, "a row stride is less than E");
    if (!known(r->dtype)) return fail(ZI_ERR_ARG, "unknown dtype %d", r->dtype);
    return ZI_OK;
}

zi_status check(const zi_combine *c) {
    if (!c) return fail(ZI_ERR_ARG, "combine is NULL");
    if (c->k < 1 || c->k > 1024) return fail(ZI_ERR_SHAPE, "k = %d: 1 .. 1024", c->k);
    if (c->T < 0 || c->T > ((int64_t)1 << 30) / c->k) return fail(ZI_ERR_SHAPE, "T = %lld: T k at most 2^30", (long long)c->T);
    if (c->R < 0 || c->R > INT32_MAX) return fail(ZI_ERR_SHAPE, "R = %lld: 0 .. 2^31 - 1 rows", (long long)c->R);
    if (c->D < 1 || c->D > INT32_MAX) return fail(ZI_ERR_SHAPE, "D = %lld: 1 .. 2^31 - 1 columns", (long long)c->D);
    if ((c->ldz != 0 && c->ldz < c->D) || (c->ldy != 0 && c->ldy < c->D) || (c->lddz != 0 && c->lddz < c->D))
        return fail(ZI_ERR_SHAPE, "a row stride is less than D");
    if (!known(c->dtype)) return fail(ZI_ERR_ARG, "unknown dtype %d", c->dtype);
    return ZI_OK;
}

// Threads that share a row: one a vector, at most a workgroup.  (Rows of 5003 fp16 on
// 128 threads, whose last turn is fuller, took a fifth longer in both directions.)
int row_threads_of(int64_t D) {
    int n = 8;
    while (n < 256 && n * 8 < D) n *= 2;
    return n;
}

}  // namespace
}  // namespace zi

using namespace zi;

extern "C" uint64_t zi_route_fwd_bytes(int64_t T, int32_t E, int32_t k) {
    (void)k;
    if (T <= kOneTokens || E < 1) return 0;
    // as many blocks as any smaller T has, so that what serves T serves those too; bytes
    // where a block has at most 128 tokens
    const int64_t blocks = ceil_div(T, 32), counts = (blocks < kMostBlocks ? blocks : kMostBlocks) * row_of(E);
    return (uint64_t)counts * (T > (int64_t)kMostBlocks * kMaskTokens ? 4 : 1);
}

extern "C" zi_status zi_route_fwd(const zi_route *r, const void *logits, int32_t *ids, float *weights, int32_t *offsets,
                                  int32_t *rows, int32_t *slots, void *workspace, uint64_t workspace_bytes, void *stream) {
    clear_error();
    const zi_status st = check(r);
    if (st != ZI_OK) return st;
    if (!offsets) return fail(ZI_ERR_ARG, "offsets are required");
    if (r->T > 0 && (!logits || !ids || !weights || !rows || !slots))
        return fail(ZI_ERR_ARG, "logits, ids, weights, rows and slots are required");
    if (!aligned(logits, size_of(r->dtype)) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(offsets, 4) ||
        !aligned(rows, 4) || !aligned(slots, 4))
        return fail(ZI_ERR_ALIGN, "a pointer is not aligned to its element");
    const uint64_t need = zi_route_fwd_bytes(r->T, r->E, r->k);
    if (need && (!workspace || workspace_bytes < need))
        return fail(ZI_ERR_BUDGET, "the workspace holds %llu B, the router needs %llu",
                    (unsigned long long)(workspace ? workspace_bytes : 0), (unsigned long long)need);
    if (!aligned(workspace, 256)) return fail(ZI_ERR_ALIGN, "the workspace is not 256-byte aligned");
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t ldl = r->ldl ? r->ldl : r->E;
    const hipError_t e = with_type(r->dtype, [&](auto type) {
        using LT = decltype(type);
        const LT *l = static_cast<const LT *>(logits);
        return with_lanes(r->E, [&](auto lanes, auto values) {
            constexpr int L = decltype(lanes)::value, V = decltype(values)::value;
            if (r->T <= kOneTokens) {
                hipLaunchKernelGGL((route_kernel<LT, L, V>), dim3(1), dim3(kOneThreads), 0, s, l, ldl, (int)r->T, r->E, r->k,
                                   r->normalize, ids, weights, offsets, rows, slots);
                return hipGetLastError();
            }
            const int64_t step = step_of(r->T, L);
            const dim3 blocks((unsigned)ceil_div(r->T, step));
            hipLaunchKernelGGL((choose_kernel<LT, L, V>), blocks, dim3(kThreads), 0, s, l, ldl, r->T, step, r->E, r->k,
                               r->normalize, ids, weights, workspace);
            const hipError_t st = hipGetLastError();
            if (st != hipSuccess) return st;
            hipLaunchKernelGGL(place_kernel, blocks, dim3(kThreads), 0, s, ids, r->T, step, r->E, r->k, workspace, offsets, rows,
                               slots);
            return hipGetLastError();
        });
    });
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "router: %s", hipGetErrorString(e));
    return ZI_OK;
}

extern "C" zi_status zi_route_bwd(const zi_route *r, const void *logits, const int32_t *ids, const float *weights,
                                  const float *dweights, void *dlogits, void *stream) {
    clear_error();
    const zi_status st = check(r);
    if (st != ZI_OK || r->T == 0) return st;
    if (!ids || !dweights || !dlogits || (r->normalize ? !weights : !logits))
        return fail(ZI_ERR_ARG, "ids, dweights, dlogits and %s are required", r->normalize ? "weights" : "logits");
    if (!aligned(logits, size_of(r->dtype)) || !aligned(dlogits, size_of(r->dtype)) || !aligned(ids, 4) || !aligned(weights, 4) ||
        !aligned(dweights, 4))
        return fail(ZI_ERR_ALIGN, "a pointer is not aligned to its element");
    hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = with_type(r->dtype, [&](auto type) {
        using LT = decltype(type);
        return with_lanes(r->E, [&](auto lanes, auto values) {
            constexpr int L = decltype(lanes)::value, V = decltype(values)::value;
            const int64_t groups = ceil_div(r->T, 256 / L);
            const dim3 grid((unsigned)(groups < 65536 ? groups : 65536));
            const LT *l = static_cast<const LT *>(logits);
            const int64_t ldl = r->ldl ? r->ldl : r->E, ldd = r->ldd ? r->ldd : r->E;
            if (r->normalize)
                hipLaunchKernelGGL((route_bwd_kernel<LT, L, V, true>), grid, dim3(256), 0, s, l, ldl, r->T, r->E, r->k, ids, weights,
                                   dweights, static_cast<LT *>(dlogits), ldd);
            else
                hipLaunchKernelGGL((route_bwd_kernel<LT, L, V, false>), grid, dim3(256), 0, s, l, ldl, r->T, r->E, r->k, ids, weights,
                                   dweights, static_cast<LT *>(dlogits), ldd);
            return hipGetLastError();
        });
    });
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "router gradient: %s", hipGetErrorString(e));
    return ZI_OK;
}

extern "C" zi_status zi_combine_fwd(const zi_combine *c, const void *Z, const int32_t *slots, const float *weights, void *Y,
                                    void *stream) {
    clear_error();
    const zi_status st = check(c);
    if (st != ZI_OK || c->T == 0) return st;
    if (!slots || !weights || !Y || (c->R > 0 && !Z)) return fail(ZI_ERR_ARG, "Z, slots, weights and Y are required");
    if (!aligned(Z, size_of(c->dtype)) || !aligned(Y, size_of(c->dtype)) || !aligned(slots, 4) || !aligned(weights, 4))
        return fail(ZI_ERR_ALIGN, "a pointer is not aligned to its element");
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int row = row_threads_of(c->D);
    const int64_t groups = ceil_div(c->T, 256 / row);
    const hipError_t e = with_type(c->dtype, [&](auto type) {
        using ZT = decltype(type);
        // few tokens: their columns are shared out too
        const int64_t parts = groups < kFewTokens ? ceil_div(c->D, 8 * row) : 1;
        hipLaunchKernelGGL((combine_fwd_kernel<ZT>), dim3((unsigned)(groups < (1 << 20) ? groups : (1 << 20)), (unsigned)(parts < 1024 ? parts : 1024)), dim3(256), 0, s,
                           static_cast<const ZT *>(Z), c->ldz ? c->ldz : c->D, c->R, slots, weights, c->T, c->D, c->k, row,
                           static_cast<ZT *>(Y), c->ldy ? c->ldy : c->D);
        return hipGetLastError();
    });
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "combination: %s", hipGetErrorString(e));
    return ZI_OK;
}

extern "C" zi_status zi_combine_bwd(const zi_combine *c, const void *dY, const void *Z, const int32_t *slots, const float *weights,
                                    void *dZ, float *dweights, void *stream) {
    clear_error();
    const zi_status st = check(c);
    if (st != ZI_OK || c->T == 0) return st;
    if (!dY || !slots || !weights || !dweights || (c->R > 0 && (!Z || !dZ)))
        return fail(ZI_ERR_ARG, "dY, Z, slots, weights, dZ and dweights are required");
    if (!aligned(Z, size_of(c->dtype)) || !aligned(dY, size_of(c->dtype)) || !aligned(dZ, size_of(c->dtype)) || !aligned(slots, 4) ||
        !aligned(weights, 4) || !aligned(dweights, 4))
        return fail(ZI_ERR_ALIGN, "a pointer is not aligned to its element");
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int row = row_threads_of(c->D);
    const int64_t groups = ceil_div(c->T, 256 / row);
    // few tokens: a workgroup a pair of rows
    const dim3 grid((unsigned)(groups < (1 << 20) ? groups : (1 << 20)), groups < kFewTokens ? (unsigned)ceil_div(c->k, KP) : 1u);
    const hipError_t e = with_type(c->dtype, [&](auto type) {
        using ZT = decltype(type);
        hipLaunchKernelGGL((combine_bwd_kernel<ZT>), grid, dim3(256), 0, s, static_cast<const ZT *>(dY), c->ldy ? c->ldy : c->D,
                           static_cast<const ZT *>(Z), c->ldz ? c->ldz : c->D, c->R, slots, weights, c->T, c->D, c->k, row,
                           static_cast<ZT *>(dZ), c->lddz ? c->lddz : c->D, dweights);
        return hipGetLastError();
    });
    if (e != hipSuccess) return fail(ZI_ERR_HIP, "combination gradient: %s", hipGetErrorString(e));
    return ZI_OK;
}
