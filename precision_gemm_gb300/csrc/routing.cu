// Routing to experts: the choice of experts and weights per token, its backward
// pass, and the experts' row lists.
#include <cfloat>

#include "layers.h"

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

// The scores of a token's experts lane, lane + 32, ...: softmax or sigmoid.  The
// softmax's sum is held in 64 bits: rounded once to 32, it does not depend on the
// order of its terms, so equal logits get equal bits whatever the layout.
template <int V>
__device__ __forceinline__ void scores(const float (&x)[V], int experts, int score, int lane, float (&p)[V]) {
    if (score == SGEMM_SCORE_SIGMOID) {
#pragma unroll
        for (int v = 0; v < V; ++v) p[v] = 1.0f / __fadd_rn(1.0f, expf(-x[v]));
        return;
    }
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, x[v]);
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    double s = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        // the largest logits give 1 also where they are infinite
        p[v] = (lane + 32 * v < experts && x[v] != -INFINITY) ? (x[v] == m ? 1.0f : expf(x[v] - m)) : 0.0f;
        s += static_cast<double>(p[v]);
    }
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    const float total = static_cast<float>(s);
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = total > 0.0f ? p[v] / total : 0.0f;
}

template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int experts, int lane, float (&x)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane + 32 * v;
        const float f = e < experts ? to_float(row[e]) : -INFINITY;
        x[v] = f != f ? -INFINITY : f;
    }
}

// One warp per token; lane l holds experts l, l + 32, ... (V of them).
template <typename T, int V>
__global__ void __launch_bounds__(128) route_kernel(int64_t tokens, int experts, int top, const T* logits, int64_t ldl,
                                                    int score, const float* balance, int groups, int group_top,
                                                    int renorm, float scale, const uint8_t* mask, float* weights,
                                                    int32_t* ids) {
    __shared__ float choice_of[4][32 * V];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + warp;
    if (t >= tokens) return;
    if (mask && mask[t] == 0) {
        if (lane < top) {
            weights[t * top + lane] = 0.0f;
            ids[t * top + lane] = -1;
        }
        return;
    }
    float x[V], p[V];
    uint32_t key[V];
    load_logits<T, V>(logits + t * ldl, experts, lane, x);
    scores<V>(x, experts, score, lane, p);
    float choice[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane + 32 * v;
        choice[v] = (balance && e < experts) ? p[v] + balance[e] : p[v];
        key[v] = e < experts ? order_key(choice[v]) : kTaken;
    }
    if (groups > 1) {
        const int per = experts / groups;
#pragma unroll
        for (int v = 0; v < V; ++v) choice_of[warp][lane + 32 * v] = choice[v];
        __syncwarp();
        uint32_t group_key = kTaken;
        if (lane < groups) {
            uint32_t k1 = kTaken, k2 = kTaken;
            float c1 = 0.0f, c2 = 0.0f;
            for (int e = lane * per; e < (lane + 1) * per; ++e) {
                const float c = choice_of[warp][e];
                const uint32_t k = order_key(c);
                if (k > k1) {
                    k2 = k1;
                    c2 = c1;
                    k1 = k;
                    c1 = c;
                } else if (k > k2) {
                    k2 = k;
                    c2 = c;
                }
            }
            group_key = order_key(c1 + c2);
        }
        uint32_t kept = 0;  // bit g: group g stays
        for (int j = 0; j < group_top; ++j) {
            const uint32_t best = __reduce_max_sync(kAll, group_key);
            const int g = __reduce_min_sync(kAll, group_key == best ? lane : 32);
            kept |= 1u << g;
            if (lane == g) group_key = kTaken;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = lane + 32 * v;
            if (e < experts && !((kept >> (e / per)) & 1u)) key[v] = kTaken;
        }
    }
    // the best key left, its lowest index; `top` times
    float my_weight = 0.0f, total = 0.0f;
    int my_id = 0;
    for (int j = 0; j < top; ++j) {
        uint32_t best = kTaken;
#pragma unroll
        for (int v = 0; v < V; ++v) best = max(best, key[v]);
        best = __reduce_max_sync(kAll, best);
        int e = 32 * V;
#pragma unroll
        for (int v = V - 1; v >= 0; --v)
            if (key[v] == best && lane + 32 * v < experts) e = lane + 32 * v;
        e = __reduce_min_sync(kAll, e);
        float w = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (lane + 32 * v == e) {
                w = p[v];
                key[v] = kTaken;
            }
        }
        w = __shfl_sync(kAll, w, e % 32);
        total += w;
        if (lane == j) {
            my_weight = w;
            my_id = e;
        }
    }
    if (renorm) my_weight = total > 0.0f ? my_weight / total : 0.0f;
    if (lane < top) {
        weights[t * top + lane] = my_weight * scale;
        ids[t * top + lane] = my_id;
    }
}

// With q_j = p[ids_j], w_j = scale q_j / (sum q)^renorm:
//   dq_j = scale (dw_j - sum(dw q) / sum(q)) / sum(q), or scale dw_j;
//   softmax: dx_e = p_e (dp_e - sum(dp p)); sigmoid: dx_e = dp_e p_e (1 - p_e).
template <typename T, int V>
__global__ void __launch_bounds__(128) route_backward_kernel(int64_t tokens, int experts, int top,
                                                             const float* dweights, const T* logits, int64_t ldl,
                                                             const int32_t* ids, int score, int renorm, float scale,
                                                             T* dlogits, int64_t lddl) {
    const int lane = threadIdx.x % 32;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32;
    if (t >= tokens) return;
    float x[V], p[V], dp[V];
    load_logits<T, V>(logits + t * ldl, experts, lane, x);
    scores<V>(x, experts, score, lane, p);
    int id = -1;
    float dw = 0.0f, q = 0.0f;
    if (lane < top) {
        id = ids[t * top + lane];
        if (id < 0 || id >= experts) id = -1;
        if (id >= 0) dw = dweights[t * top + lane] * scale;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) dp[v] = 0.0f;
    // q_j: lane id_j % 32 holds p[id_j]
    for (int j = 0; j < top; ++j) {
        const int e = __shfl_sync(kAll, id, j);
        if (e < 0) continue;
        float w = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane + 32 * v == e) w = p[v];
        w = __shfl_sync(kAll, w, e % 32);
        if (lane == j) q = w;
    }
    float dq = dw;
    if (renorm) {
        float sq = q, sdq = dw * q;
        for (int o = 16; o > 0; o >>= 1) {
            sq += __shfl_xor_sync(kAll, sq, o);
            sdq += __shfl_xor_sync(kAll, sdq, o);
        }
        dq = sq > 0.0f ? (dw - sdq / sq) / sq : 0.0f;
        if (id < 0) dq = 0.0f;
    }
    float dot = dq * q;  // sum(dp p)
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kAll, dot, o);
    for (int j = 0; j < top; ++j) {
        const int e = __shfl_sync(kAll, id, j);
        const float d = __shfl_sync(kAll, dq, j);
        if (e < 0) continue;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (lane + 32 * v == e) dp[v] += d;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = lane + 32 * v;
        if (e >= experts) continue;
        const float d = score == SGEMM_SCORE_SIGMOID ? dp[v] * p[v] * (1.0f - p[v]) : p[v] * (dp[v] - dot);
        dlogits[t * lddl + e] = from_float<T>(d);
    }
}

// ---- row lists -----------------------------------------------------------------------

constexpr int kPlanBlock = 1024;  // pairs (and threads) per block

__device__ __forceinline__ int pair_id(const int32_t* ids, int64_t pairs, int64_t i, int experts) {
    if (i >= pairs) return -1;
    const int e = ids[i];
    return (e >= 0 && e < experts) ? e : -1;
}

// hist[block][e] = the block's pairs of expert e.
__global__ void __launch_bounds__(kPlanBlock) plan_count_kernel(int64_t pairs, int experts, const int32_t* ids,
                                                                int32_t* hist) {
    __shared__ int32_t h[SGEMM_MAX_EXPERTS];
    for (int e = threadIdx.x; e < experts; e += kPlanBlock) h[e] = 0;
    __syncthreads();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kPlanBlock + threadIdx.x;
    const int e = pair_id(ids, pairs, i, experts);
    if (e >= 0) atomicAdd(&h[e], 1);
    __syncthreads();
    for (int q = threadIdx.x; q < experts; q += kPlanBlock) hist[static_cast<int64_t>(blockIdx.x) * experts + q] = h[q];
}

// Every pair's row: the expert's first row + its pairs in earlier blocks (hist),
// in earlier warps of this block, and in earlier lanes of this warp.
__global__ void __launch_bounds__(kPlanBlock) plan_place_kernel(int64_t pairs, int experts, const int32_t* ids,
                                                                const int32_t* hist, int32_t* counts,
                                                                int32_t* offsets, int32_t* rows, int32_t* slots) {
    extern __shared__ uint16_t per_warp[];  // [32][experts]
    __shared__ int32_t base[SGEMM_MAX_EXPERTS];
    __shared__ int32_t warp_sum[32];
    __shared__ int32_t used_rows;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int blocks = gridDim.x;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kPlanBlock + tid;
    for (int q = tid; q < 32 * experts; q += kPlanBlock) per_warp[q] = 0;
    __syncthreads();
    const int e = pair_id(ids, pairs, i, experts);
    const unsigned same = __match_any_sync(kAll, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) per_warp[warp * experts + e] = static_cast<uint16_t>(__popc(same));
    __syncthreads();
    // thread q < experts: expert q's totals over all blocks and over the earlier ones
    int total = 0, before = 0;
    if (tid < experts) {
        int here = 0;
        for (int w = 0; w < 32; ++w) {
            const int c = per_warp[w * experts + tid];
            per_warp[w * experts + tid] = static_cast<uint16_t>(here);
            here += c;
        }
        if (blocks == 1) {
            total = here;
        } else {
            for (int b = 0; b < blocks; ++b) {
                const int c = hist[static_cast<int64_t>(b) * experts + tid];
                if (b < static_cast<int>(blockIdx.x)) before += c;
                total += c;
            }
        }
    }
    // exclusive scan of the totals
    int scan = total;
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
    const int first = scan - total + (warp > 0 ? warp_sum[warp - 1] : 0);
    if (tid < experts) {
        base[tid] = first + before;
        if (blockIdx.x == 0) {
            counts[tid] = total;
            offsets[tid] = first;
            if (tid == experts - 1) offsets[experts] = first + total;
        }
    }
    __syncthreads();
    if (i < pairs) {
        int row = -1;
        if (e >= 0) {
            row = base[e] + per_warp[warp * experts + e] + rank;
            rows[row] = static_cast<int32_t>(i);
        }
        slots[i] = row;
        if (i >= used_rows) rows[i] = -1;  // rows that no pair takes
    }
}

template <typename T, int V>
cudaError_t run_route(int64_t tokens, int experts, int top, const void* logits, int64_t ldl, int score,
                      const float* balance, int groups, int group_top, int renorm, float scale, const uint8_t* mask,
                      float* weights, int32_t* ids, cudaStream_t st) {
    route_kernel<T, V><<<static_cast<unsigned>((tokens + 3) / 4), 128, 0, st>>>(
        tokens, experts, top, static_cast<const T*>(logits), ldl, score, balance, groups, group_top, renorm, scale,
        mask, weights, ids);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t run_route_backward(int64_t tokens, int experts, int top, const float* dweights, const void* logits,
                               int64_t ldl, const int32_t* ids, int score, int renorm, float scale, void* dlogits,
                               int64_t lddl, cudaStream_t st) {
    route_backward_kernel<T, V><<<static_cast<unsigned>((tokens + 3) / 4), 128, 0, st>>>(
        tokens, experts, top, dweights, static_cast<const T*>(logits), ldl, ids, score, renorm, scale,
        static_cast<T*>(dlogits), lddl);
    return cudaGetLastError();
}

// f<T, V> for the dtype and the values per lane that hold `experts`.
#define PG_ROUTE_DISPATCH(f, ...)                                                          \
    do {                                                                                   \
        const int per = (experts + 31) / 32;                                               \
        if (dtype == SGEMM_F32) {                                                          \
            if (per <= 1) return f<float, 1>(__VA_ARGS__);                                 \
            if (per <= 2) return f<float, 2>(__VA_ARGS__);                                 \
            if (per <= 4) return f<float, 4>(__VA_ARGS__);                                 \
            if (per <= 8) return f<float, 8>(__VA_ARGS__);                                 \
            return f<float, 16>(__VA_ARGS__);                                              \
        }                                                                                  \
        if (per <= 1) return f<bf16, 1>(__VA_ARGS__);                                      \
        if (per <= 2) return f<bf16, 2>(__VA_ARGS__);                                      \
        if (per <= 4) return f<bf16, 4>(__VA_ARGS__);                                      \
        if (per <= 8) return f<bf16, 8>(__VA_ARGS__);                                      \
        return f<bf16, 16>(__VA_ARGS__);                                                   \
    } while (0)

}  // namespace

cudaError_t launch_route(int dtype, int64_t tokens, int experts, int top, const void* logits, int64_t ldl, int score,
                         const float* balance, int groups, int group_top, int renorm, float scale,
                         const uint8_t* mask, float* weights, int32_t* ids, cudaStream_t st) {
    static_assert(SGEMM_MAX_EXPERTS <= 32 * 16, "values per lane");
    PG_ROUTE_DISPATCH(run_route, tokens, experts, top, logits, ldl, score, balance, groups, group_top, renorm, scale,
                      mask, weights, ids, st);
}

cudaError_t launch_route_backward(int dtype, int64_t tokens, int experts, int top, const float* dweights,
                                  const void* logits, int64_t ldl, const int32_t* ids, int score, int renorm,
                                  float scale, void* dlogits, int64_t lddl, cudaStream_t st) {
    PG_ROUTE_DISPATCH(run_route_backward, tokens, experts, top, dweights, logits, ldl, ids, score, renorm, scale,
                      dlogits, lddl, st);
}

static int64_t plan_blocks(int64_t pairs) { return pairs > 0 ? (pairs + kPlanBlock - 1) / kPlanBlock : 1; }

size_t plan_part_bytes(int64_t pairs, int experts) {
    const int64_t blocks = plan_blocks(pairs);
    return blocks > 1 ? static_cast<size_t>(blocks) * experts * 4 : 0;
}

int plan_launches(int64_t pairs) { return plan_blocks(pairs) > 1 ? 2 : 1; }

cudaError_t launch_expert_plan(int64_t pairs, int experts, const int32_t* ids, int32_t* counts, int32_t* offsets,
                               int32_t* rows, int32_t* slots, int32_t* part, cudaStream_t st) {
    const unsigned blocks = static_cast<unsigned>(plan_blocks(pairs));
    if (blocks > 1) plan_count_kernel<<<blocks, kPlanBlock, 0, st>>>(pairs, experts, ids, part);
    plan_place_kernel<<<blocks, kPlanBlock, 64 * experts, st>>>(pairs, experts, ids, part, counts, offsets, rows,
                                                                 slots);
    return cudaGetLastError();
}

}  // namespace pg
