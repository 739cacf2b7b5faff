// Layer norm over rows, forward and backward.
//
//     mean = sum x / n,  rstd = (sum (x - mean)^2 / n + eps)^-1/2,  h = (x - mean) rstd,
//     y = h w + b;
//     g = dy w,  dx = rstd (g - sum g / n - h sum(g h) / n) + residual,
//     dw = sum over rows of dy h,  db = sum over rows of dy.
//
// A team of W warps takes a row and keeps it in registers: one pass over memory, the
// mean first and then the squares around it, so that a mean far from zero costs no
// bits.  HBM-bound: a row is read once and its result written once.
//
// In the backward pass a thread's columns stay the same from row to row, so the sums
// for dw and db stay in its registers; a block's teams add theirs in order, and
// norm_sum_kernel adds the blocks' sums in order: equal inputs give equal bits.
// Rows too wide for the registers are read again for each of the passes.
#include <algorithm>

#include "layers.h"
#include "ptx.cuh"

namespace pg {
namespace {

constexpr int kWarp = 32;

// Column `t` of a thread's vector j: eight neighbours (VEC: 16-byte accesses), or every
// team-th column, so that a warp's single accesses fall on one line where rows start
// anywhere.
template <bool VEC>
__device__ __forceinline__ int64_t column(int tid, int team, int j, int t) {
    return VEC ? 8 * (tid + static_cast<int64_t>(team) * j) + t : tid + static_cast<int64_t>(team) * (8 * j + t);
}

// A thread's eight elements as they are stored, loaded without a use of them in between.
template <typename T>
struct Raw {
    uint4 q[sizeof(T) / 2];
    __device__ __forceinline__ float operator[](int t) const { return to_float(reinterpret_cast<const T*>(q)[t]); }
};

// Row p's elements of vector j, zero past n (n is a multiple of 8 where VEC).
template <typename T, bool VEC, bool STREAM>
__device__ __forceinline__ void fetch(const T* p, int64_t n, int tid, int team, int j, Raw<T>& v) {
    if (VEC) {
        const int64_t c = column<VEC>(tid, team, j, 0);
#pragma unroll
        for (int q = 0; q < static_cast<int>(sizeof(T)) / 2; ++q) {
            const uint4* at = reinterpret_cast<const uint4*>(p + c) + q;
            v.q[q] = c < n ? (STREAM ? __ldcs(at) : *at) : make_uint4(0, 0, 0, 0);
        }
    } else {
        T* e = reinterpret_cast<T*>(v.q);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int64_t c = column<VEC>(tid, team, j, t);
            e[t] = c < n ? p[c] : from_float<T>(0.0f);
        }
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void put(T* p, int64_t n, int tid, int team, int j, const float (&v)[8]) {
    if (VEC) {
        const int64_t c = column<VEC>(tid, team, j, 0);
        if (c < n) store8(p + c, true, 8, v);
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const int64_t c = column<VEC>(tid, team, j, t);
            if (c < n) p[c] = from_float<T>(v[t]);
        }
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sum of v over a team of `warps` warps, the same in each of its threads; `slots` holds
// a place for each warp of the block and is free again after the next call's barrier.
__device__ __forceinline__ float team_sum(float v, int warps, float* slots) {
    v = warp_sum(v);
    if (warps == 1) return v;
    const int warp = threadIdx.x / kWarp;
    if (threadIdx.x % kWarp == 0) slots[warp] = v;
    __syncthreads();
    const int first = warp / warps * warps;
    v = 0.0f;
    for (int w = 0; w < warps; ++w) v += slots[first + w];
    return v;
}

// Two sums with one barrier.
__device__ __forceinline__ float2 team_sum2(float2 v, int warps, float2* slots) {
    v = make_float2(warp_sum(v.x), warp_sum(v.y));
    if (warps == 1) return v;
    const int warp = threadIdx.x / kWarp;
    if (threadIdx.x % kWarp == 0) slots[warp] = v;
    __syncthreads();
    const int first = warp / warps * warps;
    v = make_float2(0.0f, 0.0f);
    for (int w = 0; w < warps; ++w) v = make_float2(v.x + slots[first + w].x, v.y + slots[first + w].y);
    return v;
}

struct NormParams {
    int64_t rows, n;
    const void* x;
    int64_t ldx;
    const void *w, *b;
    float eps;
    void* y;
    int64_t ldy;
    float *mean, *rstd;
    int warps;  // of a team
};

// V vectors of eight per thread.  16384 rows of 2048 float32: see the launcher.
template <typename T, bool VEC, int V, int NT>
__global__ void __launch_bounds__(NT) norm_kernel(const NormParams p) {
    __shared__ float slots[2][NT / kWarp];
    pdl_trigger();
    pdl_wait();
    const int team = p.warps * kWarp, tid = threadIdx.x % team;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / team) + threadIdx.x / team;
    const bool there = row < p.rows;
    const int64_t n = there ? p.n : 0;
    const T* x = static_cast<const T*>(p.x) + (there ? row : 0) * p.ldx;
    Raw<T> v[V];
#pragma unroll
    for (int j = 0; j < V; ++j) fetch<T, VEC, true>(x, n, tid, team, j, v[j]);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int t = 0; t < 8; ++t) sum += v[j][t];
    const float count = static_cast<float>(p.n);
    const float mean = team_sum(sum, p.warps, slots[0]) / count;
    sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float d = v[j][t] - mean;
            if (column<VEC>(tid, team, j, t) < n) sum = fmaf(d, d, sum);
        }
    const float rstd = 1.0f / sqrtf(team_sum(sum, p.warps, slots[1]) / count + p.eps);
    if (!there) return;
    if (tid == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int j = 0; j < V; ++j) {
        Raw<T> w, b;
        if (p.w) fetch<T, VEC, false>(static_cast<const T*>(p.w), n, tid, team, j, w);
        if (p.b) fetch<T, VEC, false>(static_cast<const T*>(p.b), n, tid, team, j, b);
        float o[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            const float h = (v[j][t] - mean) * rstd;
            o[t] = fmaf(h, p.w ? w[t] : 1.0f, p.b ? b[t] : 0.0f);
        }
        put<T, VEC>(y, n, tid, team, j, o);
    }
}

// Rows of any width, a block to each: three passes over the row, two of which find it in
// the caches.
template <typename T>
__global__ void __launch_bounds__(1024) norm_wide_kernel(const NormParams p) {
    __shared__ float slots[2][32];
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T *w = static_cast<const T*>(p.w), *b = static_cast<const T*>(p.b);
    float sum = 0.0f;
    for (int64_t c = threadIdx.x; c < p.n; c += 1024) sum += to_float(x[c]);
    const float count = static_cast<float>(p.n);
    const float mean = team_sum(sum, 32, slots[0]) / count;
    sum = 0.0f;
    for (int64_t c = threadIdx.x; c < p.n; c += 1024) {
        const float d = to_float(x[c]) - mean;
        sum = fmaf(d, d, sum);
    }
    const float rstd = 1.0f / sqrtf(team_sum(sum, 32, slots[1]) / count + p.eps);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + row * p.ldy;
    for (int64_t c = threadIdx.x; c < p.n; c += 1024) {
        const float h = (to_float(x[c]) - mean) * rstd;
        y[c] = from_float<T>(fmaf(h, w ? to_float(w[c]) : 1.0f, b ? to_float(b[c]) : 0.0f));
    }
}

struct NormBackwardParams {
    int64_t rows, n;
    const void* dy;
    int64_t lddy;
    const void* x;
    int64_t ldx;
    const void* w;
    const float *mean, *rstd;
    const void* residual;
    int64_t ldr;
    void* dx;
    int64_t lddx;
    float* part;  // [block][dw, db][n]
    int warps;
};

// Teams walk over rows, the next row's loads on their way while a row is worked on (AHEAD; rows of
// float32 leave no registers for it).
template <typename T, bool VEC, int V, int NT, int B, bool AHEAD>
__global__ void __launch_bounds__(NT, B) norm_backward_kernel(const NormBackwardParams p) {
    __shared__ float2 slots[2][NT / kWarp];
    extern __shared__ float sums[];  // [team][8 V][team threads], where a block has several teams
    pdl_trigger();
    pdl_wait();
    const int team = p.warps * kWarp, tid = threadIdx.x % team, teams = blockDim.x / team;
    const int64_t n = p.n, step = static_cast<int64_t>(gridDim.x) * teams;
    // every team of a block runs as many rounds, since they meet at its barriers
    const int64_t rounds = (p.rows - static_cast<int64_t>(blockIdx.x) * teams + step - 1) / step;
    int64_t row = static_cast<int64_t>(blockIdx.x) * teams + threadIdx.x / team;
    struct Row {
        Raw<T> x[V], dy[V], r[V];
        float mean, rstd;
    };
    Raw<T> w[V];
    float2 dw[V][4] = {}, db[V][4] = {};
#pragma unroll
    for (int j = 0; j < V; ++j)
        if (p.w) fetch<T, VEC, false>(static_cast<const T*>(p.w), n, tid, team, j, w[j]);
    auto load = [&](Row& to, int64_t r) {
        const int64_t there = r < p.rows ? n : 0;
        if (r >= p.rows) r = 0;
        to.mean = there ? p.mean[r] : 0.0f;
        to.rstd = there ? p.rstd[r] : 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            fetch<T, VEC, true>(static_cast<const T*>(p.x) + r * p.ldx, there, tid, team, j, to.x[j]);
            fetch<T, VEC, true>(static_cast<const T*>(p.dy) + r * p.lddy, there, tid, team, j, to.dy[j]);
            if (p.residual)
                fetch<T, VEC, true>(static_cast<const T*>(p.residual) + r * p.ldr, there, tid, team, j, to.r[j]);
        }
    };
    Row at, next;
    if (AHEAD) load(next, row);
    const float inv = 1.0f / static_cast<float>(n);
    for (int64_t round = 0; round < rounds; ++round, row += step) {
        if (AHEAD) {
            at = next;
            if (round + 1 < rounds) load(next, row + step);
        } else {
            load(at, row);
        }
        const bool there = row < p.rows;
        // two elements' (x - mean) rstd and dy w, formed again where they are needed; past the row's end
        // dy is zero, and h must not meet it as an infinity
        auto pair = [&](int j, int t, float2& h, float2& g, float2& d) {
            d = make_float2(at.dy[j][2 * t], at.dy[j][2 * t + 1]);
            const float2 x = make_float2(at.x[j][2 * t], at.x[j][2 * t + 1]);
            h = mul2(add2(x, both(-at.mean)), both(at.rstd));
            if (!VEC && (column<VEC>(tid, team, j, 2 * t) >= n || column<VEC>(tid, team, j, 2 * t + 1) >= n)) {
                if (column<VEC>(tid, team, j, 2 * t) >= n) h.x = 0.0f;
                h.y = 0.0f;
            }
            if (VEC && column<VEC>(tid, team, j, 0) >= n) h = both(0.0f);
            g = p.w ? mul2(d, make_float2(w[j][2 * t], w[j][2 * t + 1])) : d;
        };
        float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float2 h, g, d;
                pair(j, t, h, g, d);
                dw[j][t] = fma2(d, h, dw[j][t]);
                db[j][t] = add2(db[j][t], d);
                s1 = add2(s1, g);
                s2 = fma2(g, h, s2);
            }
        if (p.dx) {
            // two places for the sums, taken in turn: one barrier a round
            const float2 s = team_sum2(make_float2(s1.x + s1.y, s2.x + s2.y), p.warps, slots[round & 1]);
            if (there) {
                T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float o[8];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        float2 h, g, d;
                        pair(j, t, h, g, d);
                        const float2 v = fma2(h, both(-s.y * inv), add2(g, both(-s.x * inv)));
                        const float2 r = p.residual ? make_float2(at.r[j][2 * t], at.r[j][2 * t + 1]) : both(0.0f);
                        const float2 y = fma2(v, both(at.rstd), r);
                        o[2 * t] = y.x;
                        o[2 * t + 1] = y.y;
                    }
                    put<T, VEC>(dx, n, tid, team, j, o);
                }
            }
        }
    }
    if (!p.part) return;
    float* out = p.part + static_cast<int64_t>(blockIdx.x) * 2 * n;
#pragma unroll
    for (int which = 0; which < 2; ++which, out += n) {
        float2(&mine)[V][4] = which ? db : dw;
        auto value = [&](int j, int t) { return t & 1 ? mine[j][t / 2].y : mine[j][t / 2].x; };
        if (teams > 1) {  // the block's first team adds the others' sums in order
            __syncthreads();
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int t = 0; t < 8; ++t) sums[(threadIdx.x / team * (8 * V) + 8 * j + t) * team + tid] = value(j, t);
            __syncthreads();
            for (int q = threadIdx.x; q < 8 * V * team; q += blockDim.x) {
                const int jt = q / team;
                const int64_t c = column<VEC>(q % team, team, jt / 8, jt % 8);
                if (c >= n) continue;
                float s = 0.0f;
                for (int k = 0; k < teams; ++k) s += sums[k * (8 * V) * team + q];
                out[c] = s;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const int64_t c = column<VEC>(tid, team, j, t);
                    if (c < n) out[c] = value(j, t);
                }
        }
    }
}

// dx of rows of any width, a block to each.
template <typename T>
__global__ void __launch_bounds__(1024) norm_backward_wide_kernel(const NormBackwardParams p) {
    __shared__ float2 slots[32];
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* w = static_cast<const T*>(p.w);
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t c = threadIdx.x; c < p.n; c += 1024) {
        const float g = to_float(dy[c]) * (w ? to_float(w[c]) : 1.0f);
        s1 += g;
        s2 = fmaf(g, (to_float(x[c]) - mean) * rstd, s2);
    }
    const float inv = 1.0f / static_cast<float>(p.n);
    const float2 s = team_sum2(make_float2(s1, s2), 32, slots);
    s1 = s.x * inv;
    s2 = s.y * inv;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
    const T* r = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
    for (int64_t c = threadIdx.x; c < p.n; c += 1024) {
        const float g = to_float(dy[c]) * (w ? to_float(w[c]) : 1.0f), h = (to_float(x[c]) - mean) * rstd;
        dx[c] = from_float<T>(fmaf(rstd, g - fmaf(h, s2, s1), r ? to_float(r[c]) : 0.0f));
    }
}

// dw and db of 32 columns over a slab of rows, for rows of any width: warp l takes rows l,
// l + 8, ..., and the warps' sums are added in order.
constexpr int kSlab = 128;
template <typename T>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormBackwardParams p) {
    __shared__ float sums[2][8][kWarp];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % kWarp, l = threadIdx.x / kWarp;
    const int64_t widths = (p.n + kWarp - 1) / kWarp, slab = blockIdx.x / widths;
    const int64_t c = (blockIdx.x - slab * widths) * kWarp + lane;
    float dw = 0.0f, db = 0.0f;
    if (c < p.n) {
        const int64_t end = min((slab + 1) * kSlab, p.rows);
#pragma unroll 4
        for (int64_t r = slab * kSlab + l; r < end; r += 8) {
            const float d = to_float(static_cast<const T*>(p.dy)[r * p.lddy + c]);
            dw = fmaf(d, (to_float(static_cast<const T*>(p.x)[r * p.ldx + c]) - p.mean[r]) * p.rstd[r], dw);
            db += d;
        }
    }
    sums[0][l][lane] = dw;
    sums[1][l][lane] = db;
    __syncthreads();
    if (l < 2 && c < p.n) {
        float s = 0.0f;
        for (int q = 0; q < 8; ++q) s += sums[l][q][lane];
        p.part[(slab * 2 + l) * p.n + c] = s;
    }
}

// dw (blockIdx.y 0) and db (1): the blocks' sums, added in order by 32 warps with a 32nd of them
// each, and those in order.
__device__ __forceinline__ float sum_range(const float* part, int64_t stride, int64_t a, int64_t b) {
    float s = 0.0f;
    for (; a + 8 <= b; a += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = __ldcg(part + (a + k) * stride);
#pragma unroll
        for (int k = 0; k < 8; ++k) s += v[k];
    }
    for (; a < b; ++a) s += __ldcg(part + a * stride);
    return s;
}
template <typename T>
__global__ void __launch_bounds__(1024) norm_sum_kernel(int64_t n, int64_t blocks, const float* part, T* dw, T* db) {
    __shared__ float sums[32][kWarp + 1];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % kWarp, l = threadIdx.x / kWarp;
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kWarp + lane;
    T* out = blockIdx.y ? db : dw;
    if (!out) return;
    sums[l][lane] = c < n ? sum_range(part + blockIdx.y * n + c, 2 * n, blocks * l / 32, blocks * (l + 1) / 32) : 0.0f;
    __syncthreads();
    if (l > 0) return;
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < 32; ++q) s += sums[q][lane];
    if (c < n) out[c] = from_float<T>(s);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Warps that hold a row of n with v vectors per thread: a power of two.
int team_warps(int64_t n, int v) {
    int w = 1;
    while (static_cast<int64_t>(w) * kWarp * 8 * v < n) w *= 2;
    return w;
}

template <typename T, bool VEC, int V, int NT>
cudaError_t run_norm(NormParams p, cudaStream_t st) {
    p.warps = team_warps(p.n, V);
    const int threads = std::max(p.warps * kWarp, 256);
    return launch_kernel(true, norm_kernel<T, VEC, V, NT>,
                         dim3(static_cast<unsigned>(cdiv(p.rows, threads / (p.warps * kWarp)))), dim3(threads), 0, st, p);
}

template <typename T, bool VEC>
cudaError_t norm(const NormParams& p, int num_sms, cudaStream_t st) {
    if (p.n > 32 * kWarp * 32)
        return launch_kernel(true, norm_wide_kernel<T>, dim3(static_cast<unsigned>(p.rows)), dim3(1024), 0, st, p);
    if (p.n > 8 * kWarp * 32) return run_norm<T, VEC, 4, 1024>(p, st);
    // fewer elements per thread while the SMs are not full
    const int64_t vectors = p.rows * cdiv(p.n, 8), full = int64_t(1024) * num_sms;
    if (p.n > 8 * kWarp * 16 || vectors >= 4 * full) return run_norm<T, VEC, 4, 256>(p, st);
    if (p.n > 8 * kWarp * 8 || vectors >= 2 * full) return run_norm<T, VEC, 2, 256>(p, st);
    return run_norm<T, VEC, 1, 256>(p, st);
}

// The backward pass's shape: rows held in registers up to kHeld columns, eight of them per thread
// (sixteen of bfloat16 from 2048 on).
constexpr int64_t kHeld = 8192;
struct BackwardShape {
    int v, nt, blocks_per_sm, warps, teams;
    int64_t blocks;
};
BackwardShape backward_shape(int dtype, int64_t rows, int64_t n, int num_sms) {
    BackwardShape s{};
    s.v = dtype == SGEMM_BF16 && n > 2048 ? 2 : 1;
    s.warps = team_warps(n, s.v);
    s.nt = std::max(s.warps * kWarp, 256);
    s.blocks_per_sm = s.v == 2 ? (s.nt == 256 ? 2 : 1) : 1024 / s.nt;
    s.teams = s.nt / (s.warps * kWarp);
    s.blocks = std::min<int64_t>(cdiv(rows, s.teams), static_cast<int64_t>(s.blocks_per_sm) * num_sms);
    return s;
}

template <typename T, bool VEC, int V, int NT, int B, bool AHEAD>
cudaError_t run_backward(const NormBackwardParams& p, const BackwardShape& s, cudaStream_t st) {
    const size_t smem = s.teams > 1 && p.part ? static_cast<size_t>(s.nt) * 8 * V * 4 : 0;
    return launch_kernel(true, norm_backward_kernel<T, VEC, V, NT, B, AHEAD>, dim3(static_cast<unsigned>(s.blocks)),
                         dim3(s.nt), smem, st, p);
}

template <typename T, bool VEC>
cudaError_t norm_backward(NormBackwardParams p, const BackwardShape& s, cudaStream_t st) {
    p.warps = s.warps;
    if constexpr (std::is_same<T, bf16>::value) {
        if (s.v == 2)
            return s.nt > 256 ? run_backward<T, VEC, 2, 512, 1, true>(p, s, st)
                              : run_backward<T, VEC, 2, 256, 2, true>(p, s, st);
        return run_backward<T, VEC, 1, 256, 4, true>(p, s, st);
    } else {
        if (s.nt > 512) return run_backward<T, VEC, 1, 1024, 1, false>(p, s, st);
        return s.nt > 256 ? run_backward<T, VEC, 1, 512, 2, false>(p, s, st)
                          : run_backward<T, VEC, 1, 256, 4, false>(p, s, st);
    }
}

template <typename T>
cudaError_t backward(const NormBackwardParams& p, T* dw, T* db, int num_sms, cudaStream_t st) {
    const bool sums = dw || db;
    int64_t blocks = 0;
    cudaError_t e = cudaSuccess;
    if (p.rows > 0 && p.n <= kHeld) {
        const BackwardShape s = backward_shape(std::is_same<T, bf16>::value ? SGEMM_BF16 : SGEMM_F32, p.rows, p.n, num_sms);
        blocks = s.blocks;
        const bool vec = p.n % 8 == 0 && rows_aligned<T>(p.dy, p.lddy) && rows_aligned<T>(p.x, p.ldx) &&
                         rows_aligned<T>(p.w, 0) && rows_aligned<T>(p.residual, p.ldr) && rows_aligned<T>(p.dx, p.lddx);
        e = vec ? norm_backward<T, true>(p, s, st) : norm_backward<T, false>(p, s, st);
    } else if (p.rows > 0) {
        blocks = cdiv(p.rows, kSlab);
        if (p.dx)
            e = launch_kernel(true, norm_backward_wide_kernel<T>, dim3(static_cast<unsigned>(p.rows)), dim3(1024), 0, st, p);
        if (sums && e == cudaSuccess)
            e = launch_kernel(true, norm_columns_kernel<T>, dim3(static_cast<unsigned>(blocks * cdiv(p.n, kWarp))),
                              dim3(256), 0, st, p);
    }
    if (sums && e == cudaSuccess)
        e = launch_kernel(true, norm_sum_kernel<T>, dim3(static_cast<unsigned>(cdiv(p.n, kWarp)), 2), dim3(1024), 0, st,
                          p.n, blocks, static_cast<const float*>(p.part), dw, db);
    return e;
}

}  // namespace

cudaError_t launch_norm(int dtype, int64_t rows, int64_t n, const void* x, int64_t ldx, const void* w, const void* b,
                        float eps, void* y, int64_t ldy, float* mean, float* rstd, int num_sms, cudaStream_t st) {
    const NormParams p{rows, n, x, ldx, w, b, eps, y, ldy, mean, rstd, 1};
    auto go = [&](auto zero) {
        using T = decltype(zero);
        const bool vec = n % 8 == 0 && rows_aligned<T>(x, ldx) && rows_aligned<T>(y, ldy) && rows_aligned<T>(w, 0) &&
                         rows_aligned<T>(b, 0);
        return vec ? norm<T, true>(p, num_sms, st) : norm<T, false>(p, num_sms, st);
    };
    return dtype == SGEMM_F32 ? go(float()) : go(bf16());
}

size_t norm_part_bytes(int dtype, int64_t rows, int64_t n, int num_sms) {
    if (rows == 0) return 0;
    return static_cast<size_t>(n <= kHeld ? backward_shape(dtype, rows, n, num_sms).blocks : cdiv(rows, kSlab)) * 2 * n * 4;
}

int norm_backward_launches(int64_t rows, int64_t n, bool dx, bool sums) {
    return rows == 0 ? sums : (n <= kHeld ? 1 + sums : dx + 2 * sums);
}

cudaError_t launch_norm_backward(int dtype, int64_t rows, int64_t n, const void* dy, int64_t lddy, const void* x,
                                 int64_t ldx, const void* w, const float* mean, const float* rstd,
                                 const void* residual, int64_t ldr, void* dx, int64_t lddx, void* dw, void* db,
                                 float* part, int num_sms, cudaStream_t st) {
    const NormBackwardParams p{rows, n,        dy,  lddy, x,    ldx,                        w, mean,
                               rstd, residual, ldr, dx,   lddx, dw || db ? part : nullptr, 1};
    return dtype == SGEMM_F32
               ? backward<float>(p, static_cast<float*>(dw), static_cast<float*>(db), num_sms, st)
               : backward<bf16>(p, static_cast<bf16*>(dw), static_cast<bf16*>(db), num_sms, st);
}

}  // namespace pg
