// Routing to experts: the choice of experts and weights per token, its backward
// pass, and the experts' row lists.
#include <type_traits>

#include "layers.h"
#include "ptx.cuh"

namespace pg {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kTaken = 0, kLowest = 1;  // keys below every number's

// Unsigned keys in the order of the floats; -0 and +0 alike, NaN below -infinity.
__device__ __forceinline__ uint32_t order_key(float f) {
    if (f != f) return kLowest;
    const uint32_t b = __float_as_uint(f + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// L lanes serve one token (32 / L tokens per warp); lane l of them holds experts
// V l .. V l + V - 1, so that a token's row is read in wide loads and the lowest lane of
// equal values has the lowest index.

template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (L == 32) {
        return __reduce_max_sync(kAll, v);
    } else {
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
        return v;
    }
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}
// The lowest of the token's lanes for which `here` holds.
template <int L>
__device__ __forceinline__ int lowest_lane(bool here, int lane) {
    const uint32_t all = __ballot_sync(kAll, here) >> (lane & ~(L - 1));
    return __ffs(L == 32 ? all : all & ((1u << (L & 31)) - 1u)) - 1;
}

// a + b = s + e exactly
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
    s = __fadd_rn(a, b);
    const float t = __fsub_rn(s, a);
    e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}

// The scores of a lane's experts: softmax or sigmoid.  The softmax's sum is held in two
// floats (about 48 bits): rounded once to one, it hardly ever depends on the order of
// its terms.  (Doubles did the same at this GPU's rate for them: 33 of the 62 us of the
// backward pass at 65536 x 128.)
template <int V, int L>
__device__ __forceinline__ void scores(const float (&x)[V], int score, float (&p)[V]) {
    if (score == SGEMM_SCORE_SIGMOID) {
#pragma unroll
        for (int v = 0; v < V; ++v) p[v] = __frcp_rn(__fadd_rn(1.0f, expf(-x[v])));
        return;
    }
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, x[v]);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    float s = 0.0f, e = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        // the largest logits give 1 also where they are infinite; -infinity (also: no expert) gives 0
        p[v] = x[v] == m ? (m == -INFINITY ? 0.0f : 1.0f) : expf(x[v] - m);
        float err;
        two_sum(s, p[v], s, err);
        e += err;
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) {
        float err;
        const float os = __shfl_xor_sync(kAll, s, o), oe = __shfl_xor_sync(kAll, e, o);
        two_sum(s, os, s, err);
        e += oe + err;
    }
    const float total = s + e;
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = total > 0.0f ? p[v] / total : 0.0f;
}

// x[v]: the logits of this lane's experts, -infinity for NaN and past the last expert.
template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int experts, int first, bool vec, float (&x)[V]) {
    if (vec && V % (16 / sizeof(T)) == 0 && first + V <= experts) {
        constexpr int N = V * sizeof(T) / 16 > 0 ? V * sizeof(T) / 16 : 1;
        uint4 raw[N];
#pragma unroll
        for (int q = 0; q < N; ++q) raw[q] = reinterpret_cast<const uint4*>(row + first)[q];
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = to_float(reinterpret_cast<const T*>(raw)[v]);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = first + v < experts ? to_float(row[first + v]) : -INFINITY;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = x[v] != x[v] ? -INFINITY : x[v];
}

constexpr int kRouteWarps = 4;

// s[0] >= s[1] >= ... by Batcher's odd-even merge sort, V a power of two.
template <int V>
__device__ __forceinline__ void sort_descending(uint64_t (&s)[V]) {
#pragma unroll
    for (int p = 1; p < V; p *= 2) {
#pragma unroll
        for (int k = p; k >= 1; k /= 2) {
#pragma unroll
            for (int j = k % p; j + k < V; j += 2 * k) {
#pragma unroll
                for (int i = 0; i < k; ++i) {
                    if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
                        const uint64_t hi = s[i + j] > s[i + j + k] ? s[i + j] : s[i + j + k];
                        const uint64_t lo = s[i + j] > s[i + j + k] ? s[i + j + k] : s[i + j];
                        s[i + j] = hi;
                        s[i + j + k] = lo;
                    }
                }
            }
        }
    }
}

// Bound by its instructions: each lane sorts its keys once (with their indices below them,
// the lower index first), and a round takes the best of the lanes' heads and drops it
// from its lane.  16384 x 256, sigmoid, 4 of 8 groups, 8 experts: 19 us with the logits in
// L2, 21 from HBM (4 more when every round searched the winner's keys again).
template <typename T, int V, int L>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_kernel(int64_t tokens, int experts, int top, const T* logits, int64_t ldl, int score, const float* balance,
                 int groups, int group_top, int renorm, float scale, const uint8_t* mask, float* weights, int32_t* ids,
                 bool vec) {
    __shared__ float choice_of[kRouteWarps][L == 32 ? 32 * V : 1];
    __shared__ __align__(16) float p_of[kRouteWarps][32 * V];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, l = lane % L, first = l * V;
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp) * (32 / L) + lane / L;
    const bool some = t < tokens && (mask == nullptr || mask[t < tokens ? t : 0] != 0);
    float x[V], p[V];
    uint32_t key[V];
    load_logits<T, V>(logits + (t < tokens ? t : tokens - 1) * ldl, experts, first, vec, x);
    scores<V, L>(x, score, p);
#pragma unroll
    for (int v = 0; v < V; ++v) p_of[warp][lane * V + v] = p[v];
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const float c = balance && first + v < experts ? p[v] + balance[first + v] : p[v];
        if (L == 32 && groups > 1) choice_of[warp][L == 32 ? first + v : 0] = c;
        key[v] = first + v < experts ? order_key(c) : kTaken;
    }
    if (groups > 1) {
        const int per = experts / groups, span = per / V;  // lanes of a group
        if (per % V == 0 && (span & (span - 1)) == 0) {
            // a group's two best keys: of each lane, then over its lanes
            uint32_t k1 = kTaken, k2 = kTaken;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                k2 = max(k2, min(k1, key[v]));
                k1 = max(k1, key[v]);
            }
            for (int o = span / 2; o > 0; o >>= 1) {
                const uint32_t o1 = __shfl_xor_sync(kAll, k1, o), o2 = __shfl_xor_sync(kAll, k2, o);
                k2 = max(min(k1, o1), max(k2, o2));
                k1 = max(k1, o1);
            }
            uint32_t mine = first < experts ? order_key(key_value(k1) + key_value(k2)) : kTaken;
            bool kept = false;
            for (int j = 0; j < group_top; ++j) {
                const uint32_t best = lanes_max<L>(mine);
                const int w = lowest_lane<L>(mine == best, lane);
                if (l / span == w / span) {
                    kept = true;
                    mine = kTaken;
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = kept ? key[v] : kTaken;
        } else if (L == 32) {  // groups that do not fall on lanes: lane g goes through group g
            __syncwarp();
            uint32_t mine = kTaken;
            if (lane < groups) {
                uint32_t k1 = kTaken, k2 = kTaken;
                for (int e = lane * per; e < (lane + 1) * per; ++e) {
                    const uint32_t k = order_key(choice_of[warp][L == 32 ? e : 0]);
                    k2 = max(k2, min(k1, k));
                    k1 = max(k1, k);
                }
                mine = order_key(per > 1 ? key_value(k1) + key_value(k2) : key_value(k1));
            }
            uint32_t kept = 0;  // bit g: group g stays
            for (int j = 0; j < group_top; ++j) {
                const uint32_t best = lanes_max<32>(mine);
                const int g = lowest_lane<32>(mine == best, lane);
                kept |= 1u << g;
                if (lane == g) mine = kTaken;
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (first + v < experts && !((kept >> ((first + v) / per)) & 1u)) key[v] = kTaken;
        }
    }
    // the best head of the lanes, at the lowest lane; `top` times
    uint64_t order[V];
#pragma unroll
    for (int v = 0; v < V; ++v) order[v] = static_cast<uint64_t>(key[v]) << 32 | static_cast<uint32_t>(~(first + v));
    sort_descending<V>(order);
    int my_id = 0;
    for (int j = 0; j < top; ++j) {
        const uint32_t head = static_cast<uint32_t>(order[0] >> 32);
        const int winner = lowest_lane<L>(head == lanes_max<L>(head), lane);
        const int e = ~__shfl_sync(kAll, static_cast<int>(static_cast<uint32_t>(order[0])), winner, L);
        if (l == j) my_id = e;
        if (l == winner) {
#pragma unroll
            for (int v = 0; v + 1 < V; ++v) order[v] = order[v + 1];
            order[V - 1] = 0;
        }
    }
    float weight = l < top ? p_of[warp][(lane - l) * V + my_id] : 0.0f;
    if (renorm) {
        const float total = lanes_sum<L>(weight);
        weight = total > 0.0f ? weight / total : 0.0f;
    }
    if (l < top && t < tokens) {
        weights[t * top + l] = some ? weight * scale : 0.0f;
        ids[t * top + l] = some ? my_id : -1;
    }
}

// With q_j = p[ids_j], r_j = q_j / (sum q)^renorm, w_j = scale r_j, the gradient of a
// chosen expert's score times that score is
//   g_j = r_j scale (dw_j - sum(dw r)) renormalised, r_j scale dw_j otherwise,
// which stays finite where the scores are so small that their gradient does not, and
//   softmax: dx_e = g_e - p_e sum(g), sum(g) being 0 when renormalised;
//   sigmoid: dx_e = g_e (1 - p_e).
// The chosen scores are picked, and g placed, through shared memory.
// Reads and writes the logits once; 65536 x 128 float32: 21 us where half of them lies in
// L2 (3.2 TB/s), its softmax and shuffles as long as its bytes.
template <typename T, int V, int L>
__global__ void __launch_bounds__(32 * kRouteWarps)
    route_backward_kernel(int64_t tokens, int experts, int top, const float* dweights, const T* logits, int64_t ldl,
                          const int32_t* ids, int score, int renorm, float scale, T* dlogits, int64_t lddl, bool vec,
                          bool vec_out) {
    __shared__ __align__(16) float ps[kRouteWarps][32 * V], ds[kRouteWarps][32 * V];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, l = lane % L, first = l * V;
    const int64_t t = (static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp) * (32 / L) + lane / L;
    const bool some = t < tokens;
    float* my_p = ps[warp] + (lane - l) * V;  // the token's
    float* my_d = ds[warp] + (lane - l) * V;
    int id = -1;
    float dw = 0.0f;
    if (l < top && some) {
        id = ids[t * top + l];
        if (id < 0 || id >= experts) id = -1;
        if (id >= 0) dw = dweights[t * top + l] * scale;
    }
    float x[V], p[V];
    load_logits<T, V>(logits + (some ? t : tokens - 1) * ldl, experts, first, vec, x);
    scores<V, L>(x, score, p);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        my_p[first + v] = p[v];
        my_d[first + v] = 0.0f;
    }
    __syncwarp();
    float r = id >= 0 ? my_p[id] : 0.0f, g = dw, dot = 0.0f;
    if (renorm) {
        const float sq = lanes_sum<L>(r);
        r = sq > 0.0f ? r / sq : 0.0f;
        g = dw - lanes_sum<L>(dw * r);
    }
    g *= r;
    if (!renorm) dot = lanes_sum<L>(g);
    for (int j = 0; j < top; ++j) {  // in order: an expert may be named twice
        if (l == j && id >= 0) my_d[id] += g;
        __syncwarp();
    }
    if (!some) return;
    float d[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        d[v] = score == SGEMM_SCORE_SIGMOID ? my_d[first + v] * (1.0f - p[v]) : fmaf(-p[v], dot, my_d[first + v]);
    }
    T* out = dlogits + t * lddl + first;
    if (vec_out && V % 8 == 0 && first + V <= experts) {
#pragma unroll
        for (int v = 0; v < V; v += 8) {
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = d[(v + k) % V];
            store8(out + v, true, 8, o);
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (first + v < experts) out[v] = from_float<T>(d[v]);
    }
}

// ---- row lists -----------------------------------------------------------------------

constexpr int kPlanThreads = 1024;
constexpr int kPlanRounds = 4;                           // pairs per thread
constexpr int kPlanBlock = kPlanThreads * kPlanRounds;   // pairs per block
constexpr int kPlanLanes = kPlanThreads / 32;            // warps

__device__ __forceinline__ int pair_id(const int32_t* ids, int64_t pairs, int64_t i, int experts) {
    if (i >= pairs) return -1;
    const int e = ids[i];
    return (e >= 0 && e < experts) ? e : -1;
}

// hist[block][e] = the block's pairs of expert e.
__global__ void __launch_bounds__(kPlanThreads) plan_count_kernel(int64_t pairs, int experts, const int32_t* ids,
                                                                  int32_t* hist) {
    __shared__ int32_t h[SGEMM_MAX_EXPERTS];
    pdl_trigger();
    for (int e = threadIdx.x; e < experts; e += kPlanThreads) h[e] = 0;
    pdl_wait();
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPlanRounds; ++k) {
        const int e = pair_id(ids, pairs, static_cast<int64_t>(blockIdx.x) * kPlanBlock + k * kPlanThreads + threadIdx.x,
                              experts);
        if (e >= 0) atomicAdd(&h[e], 1);
    }
    __syncthreads();
    for (int q = threadIdx.x; q < experts; q += kPlanThreads)
        hist[static_cast<int64_t>(blockIdx.x) * experts + q] = h[q];
}

// Every pair's row: the expert's first row + its pairs in earlier blocks (hist), in
// earlier warps of this block, in earlier rounds and in earlier lanes of this warp.  A
// warp takes 128 neighbouring pairs.  Bound by its steps in a row, not by bytes: 131072
// pairs of 256 experts 11 us, the count before it 5; one block alone, without a count, 3 us.
// Every block adds up all blocks' counts, which grows with the square of the pairs: both
// kernels take 15 us at 524288 pairs of 256 experts, 188 at 4.2 million, 7.5 ms at 33 million.
__global__ void __launch_bounds__(kPlanThreads) plan_place_kernel(int64_t pairs, int experts, const int32_t* ids,
                                                                  const int32_t* hist, int32_t* counts,
                                                                  int32_t* offsets, int32_t* rows, int32_t* slots) {
    extern __shared__ uint16_t per_warp[];  // [32][experts]
    __shared__ int32_t base[SGEMM_MAX_EXPERTS];
    __shared__ int32_t sums[2][kPlanThreads];  // [total, before][part * experts + e]
    __shared__ int32_t warp_sum[32];
    __shared__ int32_t used_rows;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int blocks = gridDim.x, me = blockIdx.x;
    for (int q = tid; q < kPlanLanes * experts; q += kPlanThreads) per_warp[q] = 0;
    pdl_wait();
    __syncthreads();
    int id[kPlanRounds], rank[kPlanRounds];  // rank: among the warp's pairs of that expert
    const int64_t i0 = static_cast<int64_t>(me) * kPlanBlock + warp * (32 * kPlanRounds) + lane;
#pragma unroll
    for (int k = 0; k < kPlanRounds; ++k) id[k] = pair_id(ids, pairs, i0 + 32 * k, experts);
#pragma unroll
    for (int k = 0; k < kPlanRounds; ++k) {
        const unsigned same = __match_any_sync(kAll, id[k]);
        const int lower = __popc(same & ((1u << lane) - 1u));
        uint16_t* c = per_warp + warp * experts + (id[k] >= 0 ? id[k] : 0);
        rank[k] = id[k] >= 0 ? *c + lower : 0;
        __syncwarp();
        if (id[k] >= 0 && lower == 0) *c = static_cast<uint16_t>(rank[k] + __popc(same));
        __syncwarp();
    }
    __syncthreads();
    // expert e's totals over all blocks and over the earlier ones, shared by up to 32 threads
    const int parts = min(kPlanThreads / experts, 32), part = tid / experts, e = tid - part * experts;
    int total = 0, before = 0;
    if (part < parts && blocks > 1) {
#pragma unroll 4
        for (int b = part; b < blocks; b += parts) {
            const int c = hist[static_cast<int64_t>(b) * experts + e];
            before += b < me ? c : 0;
            total += c;
        }
        sums[0][tid] = total;
        sums[1][tid] = before;
    }
    // thread q < experts: the block's own counts become the places of each warp's first
    if (tid < experts) {
        int here = 0;
#pragma unroll 8
        for (int w = 0; w < kPlanLanes; ++w) {
            const int c = per_warp[w * experts + tid];
            per_warp[w * experts + tid] = static_cast<uint16_t>(here);
            here += c;
        }
        if (blocks == 1) total = here;
    }
    __syncthreads();
    if (tid < experts && blocks > 1)
        for (int q = 1; q < parts; ++q) {
            total += sums[0][q * experts + tid];
            before += sums[1][q * experts + tid];
        }
    // exclusive scan of the totals
    int scan = tid < experts ? total : 0;
    const int own = scan;
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kAll, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    if (warp == 0) {
        int v = warp_sum[lane];
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(kAll, v, o);
            if (lane >= o) v += u;
        }
        warp_sum[lane] = v;
        if (lane == 31) used_rows = v;
    }
    __syncthreads();
    const int first = scan - own + (warp > 0 ? warp_sum[warp - 1] : 0);
    if (tid < experts) {
        base[tid] = first + before;
        if (me == 0) {
            counts[tid] = total;
            offsets[tid] = first;
            if (tid == experts - 1) offsets[experts] = first + total;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPlanRounds; ++k) {
        const int64_t i = i0 + 32 * k;
        if (i >= pairs) continue;
        int row = -1;
        if (id[k] >= 0) {
            row = base[id[k]] + per_warp[warp * experts + id[k]] + rank[k];
            rows[row] = static_cast<int32_t>(i);
        }
        slots[i] = row;
        if (i >= used_rows) rows[i] = -1;  // rows that no pair takes
    }
}

bool logits_aligned(const void* p, int64_t ld, int size) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * size) % 16 == 0;
}

// Lanes per token and experts per lane.  Lane j keeps the j-th choice, so there are at
// least `top` lanes; groups that do not fall on whole lanes take the 32-lane form.
int route_lanes(int experts, int top, int groups) {
    for (int lanes : {8, 16}) {
        const int v = (experts + lanes - 1) / lanes;
        const int values = v <= 2 ? 2 : (v <= 4 ? 4 : 8);
        if (top > lanes || experts > 8 * lanes) continue;
        const int per = experts / groups, span = per / values;
        if (groups > 1 && (per % values != 0 || (span & (span - 1)) != 0)) continue;
        return lanes;
    }
    return 32;
}

template <typename F>
cudaError_t with_layout(int lanes, int experts, F f) {
    const int v = (experts + lanes - 1) / lanes;
    auto with_v = [&](auto l) {
        if (v <= 2) return f(l, std::integral_constant<int, 2>());
        if (v <= 4) return f(l, std::integral_constant<int, 4>());
        return f(l, std::integral_constant<int, 8>());
    };
    if (lanes == 8) return with_v(std::integral_constant<int, 8>());
    if (lanes == 16) return with_v(std::integral_constant<int, 16>());
    if (v > 8) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 16>());
    return with_v(std::integral_constant<int, 32>());
}

unsigned route_blocks(int64_t tokens, int lanes) {
    const int64_t per = kRouteWarps * (32 / lanes);
    return static_cast<unsigned>((tokens + per - 1) / per);
}

template <typename T>
cudaError_t run_route(int64_t tokens, int experts, int top, const void* logits, int64_t ldl, int score,
                      const float* balance, int groups, int group_top, int renorm, float scale, const uint8_t* mask,
                      float* weights, int32_t* ids, cudaStream_t st) {
    const int lanes = route_lanes(experts, top, groups);
    return with_layout(lanes, experts, [&](auto l, auto v) {
        return launch_kernel(true, route_kernel<T, decltype(v)::value, decltype(l)::value>,
                             dim3(route_blocks(tokens, lanes)), dim3(32 * kRouteWarps), 0, st, tokens, experts, top,
                             static_cast<const T*>(logits), ldl, score, balance, groups, group_top, renorm, scale, mask,
                             weights, ids, logits_aligned(logits, ldl, sizeof(T)));
    });
}

template <typename T>
cudaError_t run_route_backward(int64_t tokens, int experts, int top, const float* dweights, const void* logits,
                               int64_t ldl, const int32_t* ids, int score, int renorm, float scale, void* dlogits,
                               int64_t lddl, cudaStream_t st) {
    const int lanes = route_lanes(experts, top, 1);
    return with_layout(lanes, experts, [&](auto l, auto v) {
        return launch_kernel(true, route_backward_kernel<T, decltype(v)::value, decltype(l)::value>,
                             dim3(route_blocks(tokens, lanes)), dim3(32 * kRouteWarps), 0, st, tokens, experts, top,
                             dweights, static_cast<const T*>(logits), ldl, ids, score, renorm, scale,
                             static_cast<T*>(dlogits), lddl, logits_aligned(logits, ldl, sizeof(T)),
                             logits_aligned(dlogits, lddl, sizeof(T)));
    });
}

}  // namespace

cudaError_t launch_route(int dtype, int64_t tokens, int experts, int top, const void* logits, int64_t ldl, int score,
                         const float* balance, int groups, int group_top, int renorm, float scale,
                         const uint8_t* mask, float* weights, int32_t* ids, cudaStream_t st) {
    static_assert(SGEMM_MAX_EXPERTS <= 32 * 16 && SGEMM_MAX_TOP <= 32, "lanes and values per lane");
    return dtype == SGEMM_F32 ? run_route<float>(tokens, experts, top, logits, ldl, score, balance, groups, group_top,
                                                 renorm, scale, mask, weights, ids, st)
                              : run_route<bf16>(tokens, experts, top, logits, ldl, score, balance, groups, group_top,
                                                renorm, scale, mask, weights, ids, st);
}

cudaError_t launch_route_backward(int dtype, int64_t tokens, int experts, int top, const float* dweights,
                                  const void* logits, int64_t ldl, const int32_t* ids, int score, int renorm,
                                  float scale, void* dlogits, int64_t lddl, cudaStream_t st) {
    return dtype == SGEMM_F32 ? run_route_backward<float>(tokens, experts, top, dweights, logits, ldl, ids, score,
                                                          renorm, scale, dlogits, lddl, st)
                              : run_route_backward<bf16>(tokens, experts, top, dweights, logits, ldl, ids, score,
                                                         renorm, scale, dlogits, lddl, st);
}

static int64_t plan_blocks(int64_t pairs) { return pairs > 0 ? (pairs + kPlanBlock - 1) / kPlanBlock : 1; }

size_t plan_part_bytes(int64_t pairs, int experts) {
    const int64_t blocks = plan_blocks(pairs);
    return blocks > 1 ? static_cast<size_t>(blocks) * experts * 4 : 0;
}

int plan_launches(int64_t pairs) { return plan_blocks(pairs) > 1 ? 2 : 1; }

cudaError_t launch_expert_plan(int64_t pairs, int experts, const int32_t* ids, int32_t* counts, int32_t* offsets,
                               int32_t* rows, int32_t* slots, int32_t* part, cudaStream_t st) {
    static_assert(kPlanThreads >= SGEMM_MAX_EXPERTS, "a thread per expert");
    const unsigned blocks = static_cast<unsigned>(plan_blocks(pairs));
    if (blocks > 1) {
        const cudaError_t e = launch_kernel(true, plan_count_kernel, dim3(blocks), dim3(kPlanThreads), 0, st, pairs,
                                            experts, ids, part);
        if (e != cudaSuccess) return e;
    }
    return launch_kernel(true, plan_place_kernel, dim3(blocks), dim3(kPlanThreads), 2 * kPlanLanes * experts, st, pairs,
                         experts, ids, static_cast<const int32_t*>(part), counts, offsets, rows, slots);
}

}  // namespace pg
