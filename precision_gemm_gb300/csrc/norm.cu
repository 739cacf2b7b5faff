// Layer norm over rows, forward and backward.
//
//     mean = sum x / n,  rstd = (sum (x - mean)^2 / n + eps)^-1/2,  h = (x - mean) rstd,
//     y = h w + b;
//     g = dy w,  dx = rstd (g - sum g / n - h sum(g h) / n) + residual,
//     dw = sum over rows of dy h,  db = sum over rows of dy.
//
// HBM-bound: a row is read once and its result written once.  A team of warps takes a row, 64 bytes
// per thread where the row is long enough, and walks on by as many rows as there are teams; a
// row's sums cost two or three trips through a team's warps, which other teams' rows hide.  The
// next rows are on their way meanwhile, by asynchronous copies into places in shared memory that
// only the thread itself reads: no barrier is needed for them, and no registers are held.
//
// The mean is formed first and then the squares around it.  A mean m is off by a few 2^-24 m, which in
// h counts as a few 2^-24 m rstd: nothing, unless the mean is farther from zero than h's unit, 1 / rstd.
// Such a row (far_mean) takes the mean of its differences from m, which are exact, and goes on with
// what they differ from that, so that a mean far from zero costs no bits; equal values give zeros.
//
// In the backward pass a thread's columns stay the same from row to row, so the sums for dw and
// db stay in its registers; a block's teams add theirs in order, and norm_sum_kernel adds the
// blocks' sums in order: equal inputs give equal bits.  Rows too wide for that are read again for
// each of the passes.
//
// Measured (L2 cold), forward and backward without residual: 16384 x 2048 float32 51 and 69 us (5.3 and
// 5.8 TB/s), 16384 x 4096 bfloat16 56 and 84 us (4.8 TB/s), 512 x 4096 bfloat16 7 and 14 us, 1 x 4096 4 and 6 us.
// The test for far means costs the forward pass 2 to 4 % of that (rows finished again after their results are
// written: 15 %); far from zero they take 57 and 69 us.
#include <algorithm>
#include <initializer_list>
#include <utility>

#include "layers.h"
#include "ptx.cuh"

namespace pg {
namespace {

constexpr int kWarp = 32;
constexpr int kMostThreads = 512;                            // of a block
constexpr int kForwardThreads = 1024;  // of an SM: 64 registers each
constexpr int kBackwardBlocks = 2;     // of 256 threads in the backward pass, whose sums take registers

// The widest access that rows allow, in elements: G of them lie side by side and 16 bytes are the
// most.  A thread has vectors of eight elements, 8 / G accesses, each side by side with its
// neighbours': element t of vector j is column(tid, team, j, t).
template <int G>
__device__ __forceinline__ int column(int tid, int team, int j, int t) {
    return G * (tid + team * (8 / G * j + t / G)) + t % G;
}

// A thread's eight elements as they are stored, taken and put two at a time (a bfloat16 is the upper half
// of its float).
template <typename T>
struct Raw {
    uint4 q[sizeof(T) / 2];
    __device__ __forceinline__ float2 pair(int t) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(q)[t];
            return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
        } else {
            return reinterpret_cast<const float2*>(q)[t];
        }
    }
    __device__ __forceinline__ void set(int t, float2 v) {
        if constexpr (sizeof(T) == 2)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(reinterpret_cast<uint32_t*>(q)[t]) : "f"(v.y), "f"(v.x));
        else
            reinterpret_cast<float2*>(q)[t] = v;
    }
};

template <int BYTES>
struct Word;
template <>
struct Word<2> { using type = uint16_t; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<16> { using type = uint4; };

// Vector j of a row at p, zeros past n (a multiple of G).  FULL: the team's threads have n columns, and
// nothing is tested.
template <typename T, int G, bool FULL = false>
__device__ __forceinline__ void fetch(const T* p, int n, int tid, int team, int j, Raw<T>& v) {
    using W = typename Word<G * sizeof(T)>::type;
    W* to = reinterpret_cast<W*>(v.q);
#pragma unroll
    for (int a = 0; a < 8 / G; ++a) {
        const int c = column<G>(tid, team, j, G * a);
        to[a] = FULL || c < n ? *reinterpret_cast<const W*>(p + c) : W{};
    }
}
template <typename T, int G, bool FULL = false>
__device__ __forceinline__ void put(T* p, int n, int tid, int team, int j, const Raw<T>& raw) {
    using W = typename Word<G * sizeof(T)>::type;
#pragma unroll
    for (int a = 0; a < 8 / G; ++a) {
        const int c = column<G>(tid, team, j, G * a);
        if (FULL || c < n) *reinterpret_cast<W*>(p + c) = reinterpret_cast<const W*>(raw.q)[a];
    }
}

// A thread's places in shared memory: S stages of A arrays of V vectors, each access beside the
// neighbouring threads'.  Single bfloat16 elements are too small to be copied asynchronously; such
// rows are loaded where they are used.
template <typename T, int G, int V, int A, int S, int NT, bool FULL = false>
struct Stages {
    static constexpr bool ASYNC = G * sizeof(T) >= 4;
    static constexpr int BYTES = G * static_cast<int>(sizeof(T)), ACCESSES = 8 / G;
    static constexpr int ARRAY = V * ACCESSES * BYTES * NT, STAGE = A * ARRAY;  // bytes
    static constexpr size_t SHARED = ASYNC ? static_cast<size_t>(S) * STAGE : 0;
    uint8_t* base;  // this thread's
    __device__ __forceinline__ explicit Stages(uint8_t* memory, int n, int tid, int team)
        : base(memory + BYTES * threadIdx.x) {
        if constexpr (BYTES == 16 && !FULL) {  // what lies past the rows' end is zero, and no copy goes there
            using W = typename Word<BYTES>::type;
#pragma unroll
            for (int k = 0; k < V * ACCESSES; ++k)
                if (G * (tid + team * k) >= n)
                    for (int q = 0; q < S * A; ++q) *reinterpret_cast<W*>(base + q * ARRAY + k * (BYTES * NT)) = W{};
        }
    }
    // The row at p starts on its way.
    __device__ __forceinline__ void start(int stage, int array, const T* p, int n, int tid, int team) const {
        if constexpr (ASYNC) {
            const uint32_t to = smem_u32(base) + stage * STAGE + array * ARRAY;
#pragma unroll
            for (int k = 0; k < V * ACCESSES; ++k) {
                const int c = G * (tid + team * k);
                if constexpr (BYTES == 16) {
                    if (FULL || c < n)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + k * (BYTES * NT)), "l"(p + c) : "memory");
                } else {  // (a branch for each of many small copies costs more than copies of nothing)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to + k * (BYTES * NT)),
                                 "l"(c < n ? p + c : p), "n"(BYTES), "r"(c < n ? BYTES : 0)
                                 : "memory");
                }
            }
        }
    }
    // The row that was started, or the one at p where it could not be.
    __device__ __forceinline__ void read(int stage, int array, const T* p, int n, int tid, int team, int j, Raw<T>& v) const {
        if constexpr (ASYNC) {
            using W = typename Word<BYTES>::type;
            const uint8_t* from = base + stage * STAGE + array * ARRAY + j * (ACCESSES * BYTES * NT);
#pragma unroll
            for (int a = 0; a < ACCESSES; ++a) reinterpret_cast<W*>(v.q)[a] = *reinterpret_cast<const W*>(from + a * (BYTES * NT));
        } else {
            fetch<T, G, FULL>(p, n, tid, team, j, v);
        }
    }
};
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {  // all but the last N groups
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A team of `warps` warps (a power of two, 16 at most) of a block, or of 8 or 16 lanes of a warp (PARTS, whose
// kernels alone pay for it).
template <bool PARTS>
struct Team {
    int warps, threads, index, warp, lane;
    __device__ __forceinline__ Team(int w, int lanes)
        : warps(w), threads(PARTS ? lanes : w * kWarp), index(threadIdx.x / threads), warp(threadIdx.x / kWarp),
          lane(threadIdx.x % kWarp) {}
    // how far this team's row lies ahead of that of its warp's first team, which decides for the warp
    __device__ __forceinline__ int ahead() const { return PARTS ? lane / threads : 0; }
    __device__ __forceinline__ float part_sum(float v) const {
        if (threads > 8) v += __shfl_xor_sync(0xffffffffu, v, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    // a barrier of its threads alone (at most eight teams have several warps; barrier 0 is the block's)
    __device__ __forceinline__ void barrier() const {
        asm volatile("bar.sync %0, %1;" ::"r"(1 + index), "r"(warps * kWarp) : "memory");
    }
    // The sum of v over the team, the same in each thread; `slots` holds a place for each warp of the block
    // and is free again after the team's next barrier.
    __device__ __forceinline__ float sum(float v, float* slots) const {
        if (PARTS) return part_sum(v);
        v = warp_sum(v);
        if (warps == 1) return v;
        if (lane == 0) slots[warp] = v;
        barrier();
        v = slots[index * warps + (lane & (warps - 1))];
        for (int o = warps / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    // Two sums at once, one in each half of a warp.
    __device__ __forceinline__ float2 sum2(float2 v, float2* slots) const {
        if (PARTS) return make_float2(part_sum(v.x), part_sum(v.y));
        const bool upper = lane >= 16;
        float s = (upper ? v.y : v.x) + __shfl_xor_sync(0xffffffffu, upper ? v.x : v.y, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (warps > 1) {
            float* place = reinterpret_cast<float*>(slots) + (upper ? 1 : 0);
            if (lane % 16 == 0) place[2 * warp] = s;
            barrier();
            s = place[2 * (index * warps + (lane & (warps - 1)))];
            for (int o = warps / 2; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
        }
        return make_float2(__shfl_sync(0xffffffffu, s, 0), __shfl_sync(0xffffffffu, s, 16));
    }
};

// The sum over a block of 32 warps.
__device__ __forceinline__ float block_sum(float v, float* slots) {
    v = warp_sum(v);
    if (threadIdx.x % kWarp == 0) slots[threadIdx.x / kWarp] = v;
    __syncthreads();
    return warp_sum(slots[threadIdx.x % kWarp]);
}

// (var = 1 / rstd^2: nothing waits for the root)
__device__ __forceinline__ bool far_mean(float mean, float var) { return mean * mean > var; }

struct NormParams {
    int64_t rows, n;
    const void* x;
    int64_t ldx;
    const void *w, *b;
    float eps;
    void* y;
    int64_t ldy;
    float *mean, *rstd;
    int warps, lanes;  // of a team: lanes where they are no warp
    bool shared_wb;    // w and b have places in shared memory
    bool vec;          // rows too wide to be held: all in 16-byte accesses
};

// V vectors of eight per thread, S rows on their way per team.  FULL: rows fill their teams; without tests of columns
// and their branches 16384 x 4096 bfloat16 takes a sixth less time.
template <typename T, int G, int V, int S, int NT, bool FULL, bool PARTS>
__global__ void __launch_bounds__(NT, kForwardThreads / NT) norm_kernel(const NormParams p) {
    __shared__ float slots[4][NT / kWarp];
    extern __shared__ __align__(16) uint8_t memory[];
    const Team<PARTS> whole(p.warps, p.lanes);
    const int team = whole.threads, tid = threadIdx.x - whole.index * team, teams = NT / team;
    const int n = static_cast<int>(p.n);
    const Stages<T, G, V, 1, S, NT, FULL> stages(memory, n, tid, team);
    pdl_trigger();
    pdl_wait();
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    int64_t row = static_cast<int64_t>(blockIdx.x) * teams + whole.index;
    const T *w = static_cast<const T*>(p.w), *b = static_cast<const T*>(p.b);
    auto start = [&](int stage, int64_t r) {
        if (r < p.rows) stages.start(stage, 0, static_cast<const T*>(p.x) + r * p.ldx, n, tid, team);
        commit_copies();
    };
#pragma unroll
    for (int s = 0; s + 1 < S; ++s) start(s, row + s * step);
    // w and b stay in registers or, where they are too many, in shared memory: a thread reads what it
    // put there (and every team puts the same); for teams of a whole block that would leave too little for the rows
    constexpr bool KEEP = V * sizeof(T) <= 4;
    constexpr int BYTES = G * static_cast<int>(sizeof(T));
    Raw<T> kept_w[KEEP ? V : 1], kept_b[KEEP ? V : 1];
    uint8_t* const shared_w = memory + Stages<T, G, V, 1, S, NT>::SHARED + BYTES * tid;
    uint8_t* const shared_b = shared_w + BYTES * team * (V * (8 / G));
    auto place = [&](uint8_t* base, int j, int a) {
        return reinterpret_cast<typename Word<BYTES>::type*>(base + BYTES * team * (j * (8 / G) + a));
    };
#pragma unroll
    for (int j = 0; j < V; ++j) {
        Raw<T> wj, bj;
        if (w) fetch<T, G, FULL>(w, n, tid, team, j, wj);
        if (b) fetch<T, G, FULL>(b, n, tid, team, j, bj);
        if (KEEP) {
            kept_w[KEEP ? j : 0] = wj;
            kept_b[KEEP ? j : 0] = bj;
        } else if (p.shared_wb) {
#pragma unroll
            for (int a = 0; a < 8 / G; ++a) {
                *place(shared_w, j, a) = reinterpret_cast<const typename Word<BYTES>::type*>(wj.q)[a];
                *place(shared_b, j, a) = reinterpret_cast<const typename Word<BYTES>::type*>(bj.q)[a];
            }
        }
    }
    const float inv = 1.0f / static_cast<float>(n);
    int stage = 0, turn = 0;
    for (; row - whole.ahead() < p.rows; row += step) {
        const bool mine = !PARTS || row < p.rows;
        start(stage == 0 ? S - 1 : stage - 1, row + (S - 1) * step);
        wait_copies<S - 1>();
        float2 v[V][4], sum = both(0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            Raw<T> raw;
            stages.read(stage, 0, static_cast<const T*>(p.x) + (mine ? row : 0) * p.ldx, n, tid, team, j, raw);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                v[j][t] = raw.pair(t);
                sum = add2(sum, v[j][t]);
            }
        }
        // two places for each sum, taken in turn: one barrier per sum
        float mean = whole.sum(sum.x + sum.y, slots[turn]) * inv;
        // v -= by, and the sum over the row of v or (SQUARES) of v^2
        auto without = [&](float by, auto squares) {
            constexpr bool SQUARES = decltype(squares)::value;
            sum = both(0.0f);
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float2 d = v[j][t] = add2(v[j][t], both(-by));
                    if (FULL) {
                        sum = SQUARES ? fma2(d, d, sum) : add2(d, sum);
                    } else if (G == 1) {
                        if (column<G>(tid, team, j, 2 * t) < n) sum.x = SQUARES ? fmaf(d.x, d.x, sum.x) : d.x + sum.x;
                        if (column<G>(tid, team, j, 2 * t + 1) < n) sum.y = SQUARES ? fmaf(d.y, d.y, sum.y) : d.y + sum.y;
                    } else if (column<G>(tid, team, j, 2 * t / G * G) < n) {
                        sum = SQUARES ? fma2(d, d, sum) : add2(d, sum);
                    }
                }
            return sum.x + sum.y;
        };
        float var = fmaf(whole.sum(without(mean, std::true_type()), slots[turn + 1]), inv, p.eps);
        // (teams of a warp decide together, and one whose mean is near keeps its bits)
        const bool far = far_mean(mean, var);
        if (PARTS ? __any_sync(0xffffffffu, far) : far) {
            float rest = whole.sum(without(0.0f, std::false_type()), slots[turn]) / static_cast<float>(n);
            if (PARTS && !far) rest = 0.0f;
            var = fmaf(whole.sum(without(rest, std::true_type()), slots[turn + 1]), inv, p.eps);
            mean += rest;
        }
        const float rstd = 1.0f / sqrtf(var);
        turn ^= 2;
        if (tid == 0 && mine) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        T* y = static_cast<T*>(p.y) + row * p.ldy;
        auto write = [&](auto with_w, auto with_b) {
            constexpr bool W = decltype(with_w)::value, B = decltype(with_b)::value;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                Raw<T> wj, bj, o;
                if (KEEP) {
                    wj = kept_w[KEEP ? j : 0];
                    bj = kept_b[KEEP ? j : 0];
                } else if (!p.shared_wb) {
                    if (W) fetch<T, G, FULL>(w, n, tid, team, j, wj);
                    if (B) fetch<T, G, FULL>(b, n, tid, team, j, bj);
                } else {
#pragma unroll
                    for (int a = 0; a < 8 / G; ++a) {
                        if (W) reinterpret_cast<typename Word<BYTES>::type*>(wj.q)[a] = *place(shared_w, j, a);
                        if (B) reinterpret_cast<typename Word<BYTES>::type*>(bj.q)[a] = *place(shared_b, j, a);
                    }
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const float2 h = mul2(v[j][t], both(rstd));
                    o.set(t, W && B ? fma2(h, wj.pair(t), bj.pair(t))
                                    : (W ? mul2(h, wj.pair(t)) : (B ? add2(h, bj.pair(t)) : h)));
                }
                put<T, G, FULL>(y, n, tid, team, j, o);
            }
        };
        if (!mine) {
            // (this warp's other rows are there)
        } else if (w && b)
            write(std::true_type(), std::true_type());
        else if (w)
            write(std::true_type(), std::false_type());
        else if (b)
            write(std::false_type(), std::true_type());
        else
            write(std::false_type(), std::false_type());
        stage = stage + 1 == S ? 0 : stage + 1;
    }
}

// Rows of any width, a block to each: three passes over the row, two of which find it in the caches.
// E neighbouring columns of a thread at a time: eight where rows are at 16-byte boundaries, else one (2048 rows of
// 32768 bfloat16 backwards 200 us, one at a time 385; 300 of 32769, eight at a time, 81, one at a time 49).
template <typename T, int E>
__device__ __forceinline__ void load_some(const T* p, int valid, float (&v)[E]) {
    if constexpr (E == 8)
        load8(p, true, valid, v);
    else
        v[0] = to_float(*p);
}
template <typename T, int E>
__device__ __forceinline__ void store_some(T* p, int valid, const float (&v)[E]) {
    if constexpr (E == 8)
        store8(p, true, valid, v);
    else
        *p = from_float<T>(v[0]);
}
template <int E, typename F>
__device__ __forceinline__ void for_columns(int64_t n, F f) {  // f(first column, columns there)
    for (int64_t c = E * threadIdx.x; c < n; c += E * 1024) f(c, static_cast<int>(min(n - c, int64_t(E))));
}
template <typename T, int E>
__global__ void __launch_bounds__(1024) norm_wide_kernel(const NormParams p) {
    __shared__ float slots[2][32];
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T *w = static_cast<const T*>(p.w), *b = static_cast<const T*>(p.b);
    float sum = 0.0f;
    for_columns<E>(p.n, [&](int64_t c, int valid) {
        float v[E];
        load_some(x + c, valid, v);
#pragma unroll
        for (int t = 0; t < E; ++t) sum += v[t];
    });
    const float count = static_cast<float>(p.n);
    const float mean = block_sum(sum, slots[0]) / count;
    float rest = 0.0f;  // of the mean
    auto sum_of = [&](auto squares) {  // of x - mean - rest, or its squares
        float s = 0.0f;
        for_columns<E>(p.n, [&](int64_t c, int valid) {
            float v[E];
            load_some(x + c, valid, v);
#pragma unroll
            for (int t = 0; t < E; ++t) {
                const float d = v[t] - mean - rest;
                if (t < valid) s = decltype(squares)::value ? fmaf(d, d, s) : s + d;
            }
        });
        return s;
    };
    float var = block_sum(sum_of(std::true_type()), slots[1]) / count + p.eps;
    if (far_mean(mean, var)) {
        rest = block_sum(sum_of(std::false_type()), slots[0]) / count;
        var = block_sum(sum_of(std::true_type()), slots[1]) / count + p.eps;
    }
    const float rstd = 1.0f / sqrtf(var);
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[row] = mean + rest;
        if (p.rstd) p.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(p.y) + row * p.ldy;
    for_columns<E>(p.n, [&](int64_t c, int valid) {
        float v[E], g[E], a[E];
        load_some(x + c, valid, v);
        if (w) load_some(w + c, valid, g);
        if (b) load_some(b + c, valid, a);
#pragma unroll
        for (int t = 0; t < E; ++t) v[t] = fmaf((v[t] - mean - rest) * rstd, w ? g[t] : 1.0f, b ? a[t] : 0.0f);
        store_some(y + c, valid, v);
    });
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
    float* part;  // [block][dw, db][ldp]
    int64_t ldp;  // n to a multiple of four
    int warps, lanes;  // of a team
    bool vec;     // as in NormParams
};

template <typename T, int G, int V, int S, int NT, int B, bool FULL, bool PARTS>
__global__ void __launch_bounds__(NT, B)
    norm_backward_kernel(const NormBackwardParams p) {
    __shared__ float2 slots[2][NT / kWarp];
    extern __shared__ __align__(16) uint8_t memory[];
    const Team<PARTS> whole(p.warps, p.lanes);
    const int team = whole.threads, tid = threadIdx.x - whole.index * team, teams = NT / team;
    const int n = static_cast<int>(p.n);
    const Stages<T, G, V, 3, S, NT, FULL> stages(memory, n, tid, team);
    pdl_trigger();
    pdl_wait();
    const int64_t step = static_cast<int64_t>(gridDim.x) * teams;
    int64_t row = static_cast<int64_t>(blockIdx.x) * teams + whole.index;
    auto start = [&](int stage, int64_t r) {
        if (r < p.rows) {
            stages.start(stage, 0, static_cast<const T*>(p.x) + r * p.ldx, n, tid, team);
            stages.start(stage, 1, static_cast<const T*>(p.dy) + r * p.lddy, n, tid, team);
            if (p.residual) stages.start(stage, 2, static_cast<const T*>(p.residual) + r * p.ldr, n, tid, team);
        }
        commit_copies();
    };
#pragma unroll
    for (int s = 0; s + 1 < S; ++s) start(s, row + s * step);
    // w and the sums of 32 columns of a thread do not fit in its registers: bfloat16 w then comes from L1 and L2
    // (4096 rows of 16384: 137 -> 118 us; float32, with a single row on its way, 160 -> 168)
    constexpr bool KEEP = V < 4 || sizeof(T) == 4;
    float2 kept[KEEP ? V : 1][4], dw[V][4] = {}, db[V][4] = {};
    auto weights = [&](int j, float2(&w)[4]) {
        Raw<T> raw;
        if (p.w) fetch<T, G, FULL>(static_cast<const T*>(p.w), n, tid, team, j, raw);
#pragma unroll
        for (int t = 0; t < 4; ++t) w[t] = p.w ? raw.pair(t) : both(1.0f);
    };
    if constexpr (KEEP) {
#pragma unroll
        for (int j = 0; j < V; ++j) weights(j, kept[j]);
    }
    auto with_weights = [&](int j, auto f) {
        if constexpr (KEEP) {
            f(kept[j]);
        } else {
            float2 w[4];
            weights(j, w);
            f(w);
        }
    };
    float next_mean = 0.0f, next_rstd = 0.0f;
    auto statistics = [&](int64_t r) {
        next_mean = r < p.rows ? p.mean[r] : 0.0f;
        next_rstd = r < p.rows ? p.rstd[r] : 0.0f;
    };
    statistics(row);
    const float inv = 1.0f / static_cast<float>(n);
    int stage = 0, turn = 0;
    for (; row - whole.ahead() < p.rows; row += step) {
        const bool mine = !PARTS || row < p.rows;
        const int64_t at = mine ? row : 0;
        start(stage == 0 ? S - 1 : stage - 1, row + (S - 1) * step);
        const float mean = next_mean, rstd = next_rstd;
        statistics(row + step);
        wait_copies<S - 1>();
        auto read = [&](int j, Raw<T>& x, Raw<T>& dy) {
            stages.read(stage, 0, static_cast<const T*>(p.x) + at * p.ldx, n, tid, team, j, x);
            stages.read(stage, 1, static_cast<const T*>(p.dy) + at * p.lddy, n, tid, team, j, dy);
        };
        float2 s1 = both(0.0f), s2 = both(0.0f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            if (!mine) break;
            Raw<T> x, dy;
            read(j, x, dy);
            with_weights(j, [&](float2(&w)[4]) {
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    // past the row's end x and dy are zero
                    const float2 d = dy.pair(t), c = add2(x.pair(t), both(-mean)), g = mul2(d, w[t]);
                    dw[j][t] = fma2(mul2(d, both(rstd)), c, dw[j][t]);
                    db[j][t] = add2(db[j][t], d);
                    s1 = add2(s1, g);
                    s2 = fma2(g, c, s2);
                }
            });
        }
        if (p.dx) {
            // two places for the sums, taken in turn: one barrier a round
            const float2 s = whole.sum2(make_float2(s1.x + s1.y, s2.x + s2.y), slots[turn]);
            turn ^= 1;
            // dx = rstd g - rstd sum g / n - (x - mean) rstd^3 sum(g (x - mean)) / n + residual
            const float2 a = both(-rstd * (rstd * s.y * inv) * rstd), c0 = both(-rstd * (s.x * inv));
            T* dx = static_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (!mine) break;
                Raw<T> x, dy, r{};
                read(j, x, dy);
                if (p.residual)
                    stages.read(stage, 2, static_cast<const T*>(p.residual) + at * p.ldr, n, tid, team, j, r);
                Raw<T> o;
                with_weights(j, [&](float2(&w)[4]) {
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        // (w is ones where there is none, r zeros)
                        const float2 y = fma2(dy.pair(t), mul2(w[t], both(rstd)), fma2(add2(x.pair(t), both(-mean)), a, c0));
                        o.set(t, add2(y, r.pair(t)));
                    }
                });
                put<T, G, FULL>(dx, n, tid, team, j, o);
            }
        }
        stage = stage + 1 == S ? 0 : stage + 1;
    }
    if (!p.part) return;
    float* out = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.ldp;
#pragma unroll
    for (int which = 0; which < 2; ++which, out += p.ldp) {
        float2(&mine)[V][4] = which ? db : dw;
        auto value = [&](int j, int t) { return t & 1 ? mine[j][t / 2].y : mine[j][t / 2].x; };
        if (teams > 1) {  // the block's first team adds the others' sums in order
            float* sums = reinterpret_cast<float*>(memory);  // [team][8 V][team threads]
            wait_copies<0>();
            __syncthreads();
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int t = 0; t < 8; ++t) sums[(whole.index * (8 * V) + 8 * j + t) * team + tid] = value(j, t);
            __syncthreads();
            for (int q = threadIdx.x; q < 8 * V * team; q += blockDim.x) {
                const int jt = q / team;
                const int c = column<G>(q % team, team, jt / 8, jt % 8);
                if (!FULL && c >= n) continue;
                float s = 0.0f;
                for (int k = 0; k < teams; ++k) s += sums[k * (8 * V) * team + q];
                out[c] = s;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
                for (int t = 0; t < 8; t += G == 1 ? 1 : 4) {
                    const int c = column<G>(tid, team, j, t);
                    if (!FULL && c >= n) continue;
                    if constexpr (G == 1)
                        out[c] = value(j, t);
                    else
                        *reinterpret_cast<float4*>(out + c) =
                            make_float4(mine[j][t / 2].x, mine[j][t / 2].y, mine[j][t / 2 + 1].x, mine[j][t / 2 + 1].y);
                }
        }
    }
}

// dx of rows of any width, a block to each.
template <typename T, int E>
__global__ void __launch_bounds__(1024) norm_backward_wide_kernel(const NormBackwardParams p) {
    __shared__ float slots[2][32];
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + row * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + row * p.lddy;
    const T* w = static_cast<const T*>(p.w);
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    // g = dy w and h of E columns; g is zero past the row's end
    auto both_of = [&](int64_t c, int valid, float(&g)[E], float(&h)[E]) {
        float a[E];
        load_some(x + c, valid, h);
        load_some(dy + c, valid, g);
        if (w) load_some(w + c, valid, a);
#pragma unroll
        for (int t = 0; t < E; ++t) {
            if (w) g[t] *= a[t];
            h[t] = (h[t] - mean) * rstd;
        }
    };
    for_columns<E>(p.n, [&](int64_t c, int valid) {
        float g[E], h[E];
        both_of(c, valid, g, h);
#pragma unroll
        for (int t = 0; t < E; ++t) {
            s1 += g[t];
            if (t < valid) s2 = fmaf(g[t], h[t], s2);
        }
    });
    const float inv = 1.0f / static_cast<float>(p.n);
    s1 = block_sum(s1, slots[0]) * inv;
    s2 = block_sum(s2, slots[1]) * inv;
    T* dx = static_cast<T*>(p.dx) + row * p.lddx;
    const T* residual = p.residual ? static_cast<const T*>(p.residual) + row * p.ldr : nullptr;
    for_columns<E>(p.n, [&](int64_t c, int valid) {
        float g[E], h[E], r[E];
        both_of(c, valid, g, h);
        if (residual) load_some(residual + c, valid, r);
#pragma unroll
        for (int t = 0; t < E; ++t) g[t] = fmaf(rstd, g[t] - fmaf(h[t], s2, s1), residual ? r[t] : 0.0f);
        store_some(dx + c, valid, g);
    });
}

// dw and db of 32 E columns, E to a lane, over a slab of rows, for rows of any width: warp l takes rows
// l, l + 8, ..., and the warps' sums are added in order.
constexpr int kSlab = 128;
template <typename T, int E>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormBackwardParams p) {
    __shared__ float sums[8][E * kWarp];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % kWarp, l = threadIdx.x / kWarp;
    const int64_t widths = (p.n + E * kWarp - 1) / (E * kWarp), slab = blockIdx.x / widths;
    const int64_t c0 = (blockIdx.x - slab * widths) * (E * kWarp), c = c0 + E * lane;
    const int valid = static_cast<int>(min(p.n - c, int64_t(E)));
    float dw[E] = {}, db[E] = {};
    if (c < p.n) {
        const int64_t end = min((slab + 1) * kSlab, p.rows);
#pragma unroll(E == 8 ? 2 : 4)
        for (int64_t r = slab * kSlab + l; r < end; r += 8) {
            float d[E], v[E];
            load_some(static_cast<const T*>(p.dy) + r * p.lddy + c, valid, d);
            load_some(static_cast<const T*>(p.x) + r * p.ldx + c, valid, v);
            const float mean = p.mean[r], rstd = p.rstd[r];
#pragma unroll
            for (int t = 0; t < E; ++t) {
                dw[t] = fmaf(d[t], (v[t] - mean) * rstd, dw[t]);
                db[t] += d[t];
            }
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (which) __syncthreads();
#pragma unroll
        for (int t = 0; t < E; ++t) sums[l][E * lane + t] = which ? db[t] : dw[t];
        __syncthreads();
        if (threadIdx.x < E * kWarp && c0 + threadIdx.x < p.n) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) s += sums[q][threadIdx.x];
            p.part[(slab * 2 + which) * p.ldp + c0 + threadIdx.x] = s;
        }
    }
}

// dw (blockIdx.y 0) and db (1) of 32 columns, four to a thread: the blocks' sums, added in order by 32
// groups of eight threads with a 32nd of them each, and those in order.  (One column per thread of
// 1024 takes 18 us more at 16384 columns: the large blocks start one after another.)
template <typename T>
__global__ void __launch_bounds__(256) norm_sum_kernel(int64_t n, int64_t blocks, const float* part, int64_t ldp, T* dw, T* db) {
    __shared__ float4 sums[32][8];
    pdl_trigger();
    pdl_wait();
    T* out = blockIdx.y ? db : dw;
    if (!out) return;
    const int c4 = threadIdx.x % 8, l = threadIdx.x / 8;
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kWarp;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](const float4& v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
    if (c0 + 4 * c4 < ldp) {
        const float* from = part + blockIdx.y * ldp + c0 + 4 * c4;
        int64_t a = blocks * l / 32;
        const int64_t b = blocks * (l + 1) / 32;
        for (; a + 4 <= b; a += 4) {
            float4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __ldcg(reinterpret_cast<const float4*>(from + (a + k) * 2 * ldp));
#pragma unroll
            for (int k = 0; k < 4; ++k) add(v[k]);
        }
        for (; a < b; ++a) add(__ldcg(reinterpret_cast<const float4*>(from + a * 2 * ldp)));
    }
    sums[l][c4] = s;
    __syncthreads();
    if (threadIdx.x >= kWarp || c0 + threadIdx.x >= n) return;
    float total = 0.0f;
#pragma unroll
    for (int q = 0; q < 32; ++q) total += reinterpret_cast<const float*>(sums[q])[threadIdx.x];
    out[c0 + threadIdx.x] = from_float<T>(total);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Threads that hold a row of n with v vectors per thread: a power of two, whole warps or, for rows of at most
// 128, 8 or 16 lanes (65536 rows of 64 bfloat16: 6.4 us, 16 by a warp each; backwards 14.5 and 27).
int team_threads(int64_t n, int v) {
    int t = 8;
    while (static_cast<int64_t>(t) * 8 * v < n) t *= 2;
    return v > 1 && t < kWarp ? kWarp : t;
}

// Rows are held by teams: 64 bytes per thread, less where one warp then holds the row, twice as much
// where 512 threads hold it no other way.
constexpr int64_t kHeld = 16384;
struct Shape {
    int v, threads, team, teams;
    int64_t blocks;
};
template <typename T>
Shape shape_of(int64_t rows, int64_t n, int most_v, int small_blocks, int large_blocks, int num_sms) {
    Shape s{};
    s.v = 1;
    while (s.v < most_v && s.v * kWarp * 8 < n) s.v *= 2;
    while (s.v * kMostThreads * 8 < n) s.v *= 2;
    s.team = team_threads(n, s.v);
    s.threads = std::max(s.team, 256);
    s.teams = s.threads / s.team;
    s.blocks = std::min<int64_t>(cdiv(rows, s.teams), static_cast<int64_t>(s.threads > 256 ? large_blocks : small_blocks) * num_sms);
    return s;
}

// Rows of single elements take eight per thread: their addresses are many.
constexpr int most_vectors(int access, int most) { return access == 1 ? 1 : most; }
template <typename T>
constexpr int kForwardVectors = 8 / static_cast<int>(sizeof(T));
constexpr int kBackwardVectors = 2;
// f(512 threads to a block?): fewer than the most vectors per thread mean a row that a warp holds, more of them one that
// 512 threads hold no other way.
template <int V, int MOST, typename F>
cudaError_t with_threads(const Shape& s, F f) {
    if constexpr (V == MOST)
        return s.threads > 256 ? f(std::true_type()) : f(std::false_type());
    else
        return f(std::integral_constant<bool, (V > MOST)>());
}
template <typename T>
Shape backward_shape(int64_t rows, int64_t n, int access, int num_sms) {
    return shape_of<T>(rows, n, most_vectors(access, kBackwardVectors), kBackwardBlocks, 1, num_sms);
}

// The widest access (elements) that every row allows.
template <typename T>
int widest(int64_t n, std::initializer_list<std::pair<const void*, int64_t>> rows) {
    for (int g : {static_cast<int>(16 / sizeof(T)), 4}) {
        bool ok = n % g == 0;
        for (const auto& r : rows)
            ok = ok && reinterpret_cast<uintptr_t>(r.first) % (g * sizeof(T)) == 0 && r.second % g == 0;
        if (ok) return g;
    }
    return 1;
}
// f(integral_constant<widest access>)
template <typename T, typename F>
cudaError_t with_access(int g, F f) {
    if (g == 1) return f(std::integral_constant<int, 1>());
    if (sizeof(T) == 2 && g == 8) return f(std::integral_constant<int, sizeof(T) == 2 ? 8 : 4>());
    return f(std::integral_constant<int, 4>());
}

template <typename F, typename P>
cudaError_t launch_rows(F kern, std::atomic<uint64_t>& done, size_t shared, const P& p, const Shape& s, cudaStream_t st) {
    const cudaError_t e = set_smem_limit_once(done, reinterpret_cast<const void*>(kern), static_cast<int>(shared));
    if (e != cudaSuccess) return e;
    return launch_kernel(true, kern, dim3(static_cast<unsigned>(s.blocks)), dim3(s.threads), shared, st, p);
}

// Stages: an SM's shared memory holds two rows of 64 bytes per thread in the forward pass beside w and b,
// two of each of the backward pass's three matrices; more of less, and of twice as much one row.
template <typename T, int G, int V, int S, int NT>
cudaError_t run_norm(NormParams p, Shape s, int num_sms, cudaStream_t st) {
    static std::atomic<uint64_t> done[3];
    constexpr int VECTOR = 8 * V * static_cast<int>(sizeof(T));  // bytes of a thread
    s.teams = NT / s.team;
    s.blocks = std::min<int64_t>(cdiv(p.rows, s.teams), static_cast<int64_t>(kForwardThreads / NT) * num_sms);
    p.shared_wb = VECTOR > 32 && s.teams > 1;
    auto kern = norm_kernel<T, G, V, S, NT, false, false>;
    const bool parts = s.team < kWarp, full = !parts && G * sizeof(T) == 16 && p.n == static_cast<int64_t>(8 * V) * s.team;
    if constexpr (G * sizeof(T) == 16)
        if (full) kern = norm_kernel<T, G, V, S, NT, true, false>;
    if constexpr (V == 1 && NT == 256)
        if (parts) kern = norm_kernel<T, G, V, S, NT, false, true>;
    const size_t most = Stages<T, G, V, 1, S, NT>::SHARED + (VECTOR > 32 ? VECTOR * NT : 0);
    const cudaError_t e =
        set_smem_limit_once(done[parts ? 2 : full], reinterpret_cast<const void*>(kern), static_cast<int>(most));
    if (e != cudaSuccess) return e;
    const size_t smem = Stages<T, G, V, 1, S, NT>::SHARED + (p.shared_wb ? 2 * VECTOR * s.team : 0);
    return launch_kernel(true, kern, dim3(static_cast<unsigned>(s.blocks)), dim3(NT), smem, st, p);
}
// 64 bytes per thread: blocks of 512, so that more teams share w and b.
template <typename T, int G, int V>
cudaError_t run_norm(const NormParams& p, const Shape& s, int num_sms, cudaStream_t st) {
    constexpr int VECTOR = 8 * V * static_cast<int>(sizeof(T)), S = VECTOR > 64 ? 1 : (VECTOR == 64 ? 2 : 6);
    return with_threads<V, most_vectors(G, kForwardVectors<T>)>(s, [&](auto many) {
        constexpr int NT = decltype(many)::value || VECTOR > 32 ? kMostThreads : 256;
        return run_norm<T, G, V, S, NT>(p, s, num_sms, st);
    });
}
template <typename T, int G, int V, bool FULL, bool PARTS>
cudaError_t run_backward(const NormBackwardParams& p, const Shape& s, cudaStream_t st) {
    constexpr int BYTES = 8 * V * static_cast<int>(sizeof(T)), S = BYTES > 64 ? 1 : 128 / BYTES;
    return with_threads<V, most_vectors(G, kBackwardVectors)>(s, [&](auto many) {
        constexpr bool MANY = decltype(many)::value;
        constexpr int NT = MANY ? kMostThreads : 256, B = MANY ? 1 : kBackwardBlocks;
        if constexpr (MANY && PARTS) {
            return cudaErrorInvalidValue;  // (parts of a warp hold their rows)
        } else {
            static std::atomic<uint64_t> done{0};
            // teams of fewer than all threads add their sums in the same memory
            const size_t sums = MANY ? 0 : static_cast<size_t>(NT) * 8 * V * 4;
            return launch_rows(norm_backward_kernel<T, G, V, S, NT, B, FULL, PARTS>, done,
                               std::max(Stages<T, G, V, 3, S, NT>::SHARED, sums), p, s, st);
        }
    });
}
// Without tests of columns where 32 columns per thread fill their teams: 4096 x 16384 with residual 128 us instead of
// 174 (bfloat16), 194 instead of 233 (float32).  Fewer columns per thread run better with the tests (16384 x 4096 bfloat16
// 92 us, 116 without), whose branches keep the loads of a row's parts apart.
template <typename T, int G, int V>
cudaError_t run_backward(const NormBackwardParams& p, const Shape& s, cudaStream_t st) {
    if constexpr (G * sizeof(T) == 16 && V == 4)
        if (p.n == static_cast<int64_t>(8 * V) * s.team) return run_backward<T, G, V, true, false>(p, s, st);
    if constexpr (V == 1)
        if (s.team < kWarp) return run_backward<T, G, V, false, true>(p, s, st);
    return run_backward<T, G, V, false, false>(p, s, st);
}
// f(widest access, vectors per thread) as constants
template <typename T, typename F>
cudaError_t with_shape(int g, int v, F f) {
    return with_access<T>(g, [&](auto access) {
        if (v == 1) return f(access, std::integral_constant<int, 1>());
        if (v == 2) return f(access, std::integral_constant<int, 2>());
        return f(access, std::integral_constant<int, 4>());
    });
}

template <typename T>
cudaError_t norm(NormParams p, int num_sms, cudaStream_t st) {
    if (p.n > kHeld)
        return launch_kernel(true, p.vec ? norm_wide_kernel<T, 8> : norm_wide_kernel<T, 1>, dim3(static_cast<unsigned>(p.rows)), dim3(1024), 0, st, p);
    const int access = widest<T>(p.n, {{p.x, p.ldx}, {p.y, p.ldy}, {p.w, 0}, {p.b, 0}});
    const Shape s = shape_of<T>(p.rows, p.n, most_vectors(access, kForwardVectors<T>), kForwardThreads / 256,
                                kForwardThreads / kMostThreads, num_sms);
    p.warps = std::max(s.team / kWarp, 1);
    p.lanes = s.team;
    return with_shape<T>(access, s.v, [&](auto g, auto v) {
        return run_norm<T, decltype(g)::value, decltype(v)::value>(p, s, num_sms, st);
    });
}
template <typename T>
cudaError_t norm_backward(NormBackwardParams p, const Shape& s, int access, cudaStream_t st) {
    p.warps = std::max(s.team / kWarp, 1);
    p.lanes = s.team;
    return with_shape<T>(access, s.v, [&](auto g, auto v) {
        return run_backward<T, decltype(g)::value, decltype(v)::value>(p, s, st);
    });
}

template <typename T>
cudaError_t backward(const NormBackwardParams& p, T* dw, T* db, int num_sms, cudaStream_t st) {
    const bool sums = dw || db;
    int64_t blocks = 0;
    cudaError_t e = cudaSuccess;
    if (p.rows > 0 && p.n <= kHeld) {
        const int access = widest<T>(p.n, {{p.dy, p.lddy}, {p.x, p.ldx}, {p.w, 0}, {p.residual, p.ldr}, {p.dx, p.lddx}});
        const Shape s = backward_shape<T>(p.rows, p.n, access, num_sms);
        blocks = s.blocks;
        e = norm_backward<T>(p, s, access, st);
    } else if (p.rows > 0) {
        blocks = cdiv(p.rows, kSlab);
        if (sums)  // first: dx may lie over x or dy
            e = launch_kernel(true, p.vec ? norm_columns_kernel<T, 8> : norm_columns_kernel<T, 1>,
                              dim3(static_cast<unsigned>(blocks * cdiv(p.n, (p.vec ? 8 : 1) * kWarp))),
                              dim3(256), 0, st, p);
        if (p.dx && e == cudaSuccess)
            e = launch_kernel(true, p.vec ? norm_backward_wide_kernel<T, 8> : norm_backward_wide_kernel<T, 1>,
                              dim3(static_cast<unsigned>(p.rows)), dim3(1024), 0, st, p);
    }
    if (sums && e == cudaSuccess)
        e = launch_kernel(true, norm_sum_kernel<T>, dim3(static_cast<unsigned>(cdiv(p.n, kWarp)), 2), dim3(256), 0, st,
                          p.n, blocks, static_cast<const float*>(p.part), p.ldp, dw, db);
    return e;
}

}  // namespace

// Rows and vectors at 16-byte boundaries.
static bool all_aligned(int dtype, std::initializer_list<std::pair<const void*, int64_t>> rows) {
    for (const auto& r : rows)
        if (!(dtype == SGEMM_F32 ? rows_aligned<float>(r.first, r.second) : rows_aligned<bf16>(r.first, r.second))) return false;
    return true;
}

cudaError_t launch_norm(int dtype, int64_t rows, int64_t n, const void* x, int64_t ldx, const void* w, const void* b,
                        float eps, void* y, int64_t ldy, float* mean, float* rstd, int num_sms, cudaStream_t st) {
    const NormParams p{rows, n,    x,    ldx, w,     b, eps, y, ldy,
                       mean, rstd, 1,    0,    false, all_aligned(dtype, {{x, ldx}, {y, ldy}, {w, 0}, {b, 0}})};
    return dtype == SGEMM_F32 ? norm<float>(p, num_sms, st) : norm<bf16>(p, num_sms, st);
}

// (whatever the rows' alignment turns out to be)
size_t norm_part_bytes(int64_t rows, int64_t n, int num_sms) {
    if (rows == 0) return 0;
    int64_t blocks = cdiv(rows, kSlab);
    if (n <= kHeld) blocks = std::min<int64_t>(rows, int64_t(kBackwardBlocks) * num_sms);
    return static_cast<size_t>(blocks) * 2 * (cdiv(n, 4) * 4) * 4;
}

int norm_backward_launches(int64_t rows, int64_t n, bool dx, bool sums) {
    return rows == 0 ? sums : (n <= kHeld ? 1 + sums : dx + 2 * sums);
}

cudaError_t launch_norm_backward(int dtype, int64_t rows, int64_t n, const void* dy, int64_t lddy, const void* x,
                                 int64_t ldx, const void* w, const float* mean, const float* rstd,
                                 const void* residual, int64_t ldr, void* dx, int64_t lddx, void* dw, void* db,
                                 float* part, int num_sms, cudaStream_t st) {
    const NormBackwardParams p{rows, n,        dy,  lddy, x,    ldx,                        w, mean,
                               rstd, residual, ldr, dx,   lddx, dw || db ? part : nullptr, cdiv(n, 4) * 4, 1, 0,
                               all_aligned(dtype, {{dy, lddy}, {x, ldx}, {w, 0}, {residual, ldr}, {dx, lddx}})};
    return dtype == SGEMM_F32
               ? backward<float>(p, static_cast<float*>(dw), static_cast<float*>(db), num_sms, st)
               : backward<bf16>(p, static_cast<bf16*>(dw), static_cast<bf16*>(db), num_sms, st);
}

}  // namespace pg
