// Row-wise kernels of the layer calls: the activation's backward pass with the
// bias gradient, and the weighted sum of a token's expert rows in both directions.
#include "layers.h"
#include "ptx.cuh"

namespace pg {
namespace {

constexpr int kWidth = 256;  // columns per block of the activation's backward pass: 32 threads of eight

// Its rows: 128, so that a thread has sixteen to load, or 32 while that makes fewer than
// four blocks per SM (1300 x 1000 float32 13 -> 9 us).
int slab_rows(int64_t rows, int64_t n, int num_sms) {
    return ((rows + 127) / 128) * ((n + kWidth - 1) / kWidth) >= int64_t(4) * num_sms ? 128 : 32;
}

// dz = dy * act'(z) for a slab of rows x 256 columns, and the slab's column sums per
// group: a slab's rows may belong to several groups, whose sums go to the slots
// slab + g of part ((slabs + groups) x n) -- slab + g grows with every new slab and
// with every new group, so no two sums share a slot.  Thread (l, c) takes rows l, l + 8,
// ... of a group and eight columns; the eight threads of a column add up in order.
// HBM-bound: reads dy and z, writes dz (8192 x 8192 bfloat16, gelu: 68 us, 5.9 TB/s), and
// near its instructions: packed arithmetic took 32768 x 1024 of 64 experts from 50 to 45 us,
// four blocks per SM of two rows' loads each, instead of three of four rows', to 38.
template <typename T, int PARTS>
__global__ void __launch_bounds__(256, 4) dact_kernel(int64_t rows, int64_t n, const T* dy, int64_t lddy, const T* z,
                                                   int64_t ldz, int act, bf16* dz, int64_t lddz, int groups,
                                                   const int32_t* offsets, float* part, int slab_size, bool vec) {
    __shared__ float sums[8][kWidth + 8];
    pdl_trigger();
    pdl_wait();
    const int64_t widths = (n + kWidth - 1) / kWidth, slab = blockIdx.x / widths;
    const int64_t c0 = (blockIdx.x - slab * widths) * kWidth, c = c0 + 8 * (threadIdx.x % 32);
    const int l = threadIdx.x / 32;
    const int valid = static_cast<int>(n - c < 8 ? n - c : 8);  // <= 0: no columns here
    const int r0 = static_cast<int>(slab * slab_size);
    const int r1 = static_cast<int>(rows - r0 < slab_size ? rows : r0 + slab_size);
    int g = 0, first = 0, end = static_cast<int>(rows);
    if (offsets) {  // the last group that starts at or before r0: an empty one or the slab's first
        int before = 0;
        for (int q = 0; q < groups; q += 256)
            before += __syncthreads_count(q + static_cast<int>(threadIdx.x) < groups &&
                                          offsets[min(q + static_cast<int>(threadIdx.x), groups - 1)] <= r0);
        g = max(before - 1, 0);
    }
    for (; g < groups; ++g) {
        if (offsets) expert_rows(offsets, g, static_cast<int>(rows), first, end);
        const int a = max(first, r0), b = min(end, r1);
        if (first >= r1) break;
        if (a >= b) continue;
        float2 sum[4] = {};
        auto one = [&](auto f, int64_t r, float(&d)[8], const float(&s)[8]) {
            constexpr int ACT = decltype(f)::value;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                float2 v = make_float2(d[2 * t], d[2 * t + 1]);
                if (ACT != SGEMM_ACT_NONE)
                    v = mul2(v, act_derivative2<ACT, PARTS == 1>(make_float2(s[2 * t], s[2 * t + 1])));
                sum[t] = add2(sum[t], v);
                d[2 * t] = v.x;
                d[2 * t + 1] = v.y;
            }
            if (dz) store_parts8<PARTS>(dz + r * lddz + c, rows * lddz, d);
        };
        // The choices are made outside the row loops, which then have R rows' loads in flight.
        if (valid > 0) {
            with_act(act, [&](auto f) {
                constexpr bool Z = decltype(f)::value != SGEMM_ACT_NONE;
                constexpr int N = sizeof(T) / 2, R = 2 / N;  // 16-byte words of eight elements; rows
                int64_t r = a + l;
                if (vec && valid == 8) {
                    for (; r + 8 * (R - 1) < b; r += 8 * R) {
                        uint4 d[R][N], s[R][N];
#pragma unroll
                        for (int k = 0; k < R; ++k)
#pragma unroll
                            for (int q = 0; q < N; ++q) {
                                d[k][q] = __ldcs(reinterpret_cast<const uint4*>(dy + (r + 8 * k) * lddy + c) + q);
                                if (Z) s[k][q] = __ldcs(reinterpret_cast<const uint4*>(z + (r + 8 * k) * ldz + c) + q);
                            }
#pragma unroll
                        for (int k = 0; k < R; ++k) {
                            float df[8], sf[8];
#pragma unroll
                            for (int t = 0; t < 8; ++t) {
                                df[t] = to_float(reinterpret_cast<const T*>(d[k])[t]);
                                if (Z) sf[t] = to_float(reinterpret_cast<const T*>(s[k])[t]);
                            }
                            one(f, r + 8 * k, df, sf);
                        }
                    }
                }
#pragma unroll 1
                for (; r < b; r += 8) {
                    float df[8], sf[8];
                    load8(dy + r * lddy + c, vec, valid, df);
                    if (Z) load8(z + r * ldz + c, vec, valid, sf);
                    one(f, r, df, sf);
                }
            });
        }
        if (part) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                sums[l][8 * (threadIdx.x % 32) + 2 * t] = sum[t].x;
                sums[l][8 * (threadIdx.x % 32) + 2 * t + 1] = sum[t].y;
            }
            __syncthreads();
            const int64_t col = c0 + threadIdx.x;
            if (col < n) {
                float s = 0.0f;
#pragma unroll
                for (int q = 0; q < 8; ++q) s += sums[q][threadIdx.x];
                part[(slab + g) * n + col] = s;
            }
            __syncthreads();
        }
    }
}

// dz = [dy v act'(g), dy act(g)] for a slab of rows x 256 columns of z = [g v], and the slab's
// sums of its 2 n columns in part (slabs x 2 n), with the threads laid out as in dact_kernel: thread
// (l, c) takes rows l, l + 8, ... and eight columns, neighbouring ones where all rows are whole eights at
// 16-byte boundaries (VEC), else every 32nd, so that a warp's single elements are neighbours.
// dz null: the sums alone.
//
// For bfloat16 dz is rounded to it, the type of the products' operands: dx and dw then carry two
// roundings, 0.0023 of their size where one is 0.0017.  A second part of dz would keep it and double both
// products' time.  The sums take dz unrounded.
//
// HBM-bound: reads dy and z, writes dz.  bfloat16 runs best with as many threads as fit (8192 x 4096, gelu, with
// dbias: 63 us, 5.3 TB/s; 79 with half as many of two rows' loads each), float32, whose dz are three parts,
// with half of them (147 us, 5.5 TB/s; 163).  The sums alone take 41 us of the 63.
template <typename T, int PARTS, bool VEC>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2)
    dgate_kernel(int64_t rows, int64_t n, const T* dy, int64_t lddy, const T* z, int64_t ldz, int act, bf16* dz,
                 int64_t lddz, float* part, int slab_size) {
    __shared__ float sums[8][kWidth + 8];
    pdl_trigger();
    pdl_wait();
    const int64_t widths = (n + kWidth - 1) / kWidth, slab = blockIdx.x / widths;
    const int64_t c0 = (blockIdx.x - slab * widths) * kWidth;
    const int lane = threadIdx.x % 32, l = threadIdx.x / 32;
    auto column = [&](int t) { return VEC ? 8 * lane + t : lane + 32 * t; };
    const int width = static_cast<int>(min(n - c0, int64_t(kWidth)));
    const int64_t r0 = slab * slab_size, r1 = rows - r0 < slab_size ? rows : r0 + slab_size;
    dy += c0;
    z += c0;
    if (dz) dz += c0;
    float sum[2][8] = {};
    auto one = [&](auto f, int64_t r, const float(&d)[8], const float(&g)[8], const float(&v)[8]) {
        float dg[8], dv[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            float value, slope;
            act_both<decltype(f)::value, PARTS == 1>(g[t], value, slope);
            dg[t] = d[t] * v[t] * slope;
            dv[t] = d[t] * value;
            sum[0][t] += dg[t];
            sum[1][t] += dv[t];
        }
        if (!dz) return;
        bf16* at = dz + r * lddz + column(0);
        if (VEC) {
            store_parts8<PARTS>(at, rows * lddz, dg);
            store_parts8<PARTS>(at + n, rows * lddz, dv);
        } else {
            uint32_t a[PARTS][4], b[PARTS][4];
            split8<PARTS>(dg, a);
            split8<PARTS>(dv, b);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                if (column(t) >= width) break;
#pragma unroll
                for (int q = 0; q < PARTS; ++q) {
                    at[q * rows * lddz + 32 * t] = __ushort_as_bfloat16(static_cast<uint16_t>(a[q][t / 2] >> (16 * (t % 2))));
                    at[q * rows * lddz + n + 32 * t] = __ushort_as_bfloat16(static_cast<uint16_t>(b[q][t / 2] >> (16 * (t % 2))));
                }
            }
        }
    };
    if (column(0) < width) {
        with_act(act, [&](auto f) {
            auto load = [&](const T* from, float(&v)[8]) {
                if (VEC) {
                    constexpr int N = sizeof(T) / 2;  // 16-byte words of eight elements
                    uint4 raw[N];
#pragma unroll
                    for (int q = 0; q < N; ++q) raw[q] = __ldcs(reinterpret_cast<const uint4*>(from + column(0)) + q);
#pragma unroll
                    for (int t = 0; t < 8; ++t) v[t] = to_float(reinterpret_cast<const T*>(raw)[t]);
                } else {
#pragma unroll
                    for (int t = 0; t < 8; ++t) v[t] = column(t) < width ? to_float(from[column(t)]) : 0.0f;
                }
            };
#pragma unroll 1
            for (int64_t r = r0 + l; r < r1; r += 8) {
                float df[8], gf[8], vf[8];
                load(dy + r * lddy, df);
                load(z + r * ldz, gf);
                load(z + r * ldz + n, vf);
                one(f, r, df, gf, vf);
            }
        });
    }
    if (!part) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int t = 0; t < 8; ++t) sums[l][column(t)] = sum[which][t];
        __syncthreads();
        const int64_t col = c0 + threadIdx.x;
        if (col < n) {
            float s = 0.0f;
#pragma unroll
            for (int q = 0; q < 8; ++q) s += sums[q][threadIdx.x];
            part[slab * 2 * n + which * n + col] = s;
        }
        __syncthreads();
    }
}

// dbias[g][c] = the sums of group g's slabs: 8 threads per column take every eighth,
// and their sums are added in order.
template <typename T>
__global__ void __launch_bounds__(256) dbias_kernel(int64_t rows, int64_t n, const int32_t* offsets,
                                                    const float* part, T* dbias, int slab_size) {
    __shared__ float sums[8][33];
    pdl_trigger();
    pdl_wait();
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;
    const int g = blockIdx.y, l = threadIdx.x / 32;
    int first = 0, end = static_cast<int>(rows);
    if (offsets) expert_rows(offsets, g, static_cast<int>(rows), first, end);
    float sum = 0.0f;
    if (c < n && end > first) {
#pragma unroll 4
        for (int s = first / slab_size + l; s <= (end - 1) / slab_size; s += 8) sum += part[(static_cast<int64_t>(s) + g) * n + c];
    }
    sums[l][threadIdx.x % 32] = sum;
    __syncthreads();
    if (l == 0 && c < n) {
        for (int q = 1; q < 8; ++q) sum += sums[q][threadIdx.x];
        dbias[g * n + c] = from_float<T>(sum);
    }
}

// Eight elements as they were loaded.
template <typename T>
__device__ __forceinline__ void load_raw8(const T* p, uint4 (&raw)[sizeof(T) / 2]) {
#pragma unroll
    for (int q = 0; q < static_cast<int>(sizeof(T)) / 2; ++q) raw[q] = __ldcs(reinterpret_cast<const uint4*>(p) + q);
}

// `share` warps of a block take one token's columns, 256 at a time; a lane takes eight of
// them, with the loads of R rows in flight.  The token's slots and weights are read once,
// one by each lane.  HBM-bound on the rows (32768 rows of 2048 to 4096
// tokens: bfloat16 27 us, 5.5 TB/s, float32 41 us; 45 and 48 with a thread per eight columns,
// each reading the slots itself).
template <typename T, typename TX>
__global__ void __launch_bounds__(256) combine_kernel(int64_t tokens, int top, int64_t n, const TX* x, int64_t ldx,
                                                      const int32_t* slots, const float* weights, const T* residual,
                                                      int64_t ldr, T* y, int64_t ldy, bool vec, int share) {
    constexpr int N = sizeof(TX) / 2, R = 8 / N;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (8 / share) + warp / share, rows = tokens * top;
    if (t >= tokens) return;
    int slot = -1;
    float weight = 0.0f;
    if (lane < top) {
        slot = slots[t * top + lane];
        if (slot >= rows) slot = -1;
        if (slot >= 0) weight = weights ? weights[t * top + lane] : 1.0f;
    }
    for (int64_t c = (static_cast<int64_t>(blockIdx.y) * share + warp % share) * 256 + 8 * lane; c - 8 * lane < n;
         c += static_cast<int64_t>(gridDim.y) * share * 256) {
        const int64_t left = n - c;  // <= 0: no columns here
        const int valid = static_cast<int>(left < 8 ? left : 8);
        float sum[8] = {};
        for (int j0 = 0; j0 < top; j0 += R) {
            uint4 raw[R][N];
            float w[R];
#pragma unroll
            for (int j = 0; j < R; ++j) {
                const int64_t s = __shfl_sync(0xffffffffu, slot, (j0 + j) & 31);
                w[j] = __shfl_sync(0xffffffffu, weight, (j0 + j) & 31);
                const bool some = j0 + j < top && s >= 0;
                if (!some) w[j] = 0.0f;
#pragma unroll
                for (int q = 0; q < N; ++q) raw[j][q] = make_uint4(0, 0, 0, 0);
                if (some && vec && valid == 8) {
                    load_raw8(x + s * ldx + c, raw[j]);
                } else if (some) {
                    TX* e = reinterpret_cast<TX*>(raw[j]);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < valid) e[k] = x[s * ldx + c + k];
                }
            }
#pragma unroll
            for (int j = 0; j < R; ++j)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    sum[k] = fmaf(w[j], to_float(reinterpret_cast<const TX*>(raw[j])[k]), sum[k]);
        }
        if (residual && valid > 0) {
            float r[8];
            load8(residual + t * ldr + c, vec, valid, r);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] += r[k];
        }
        if (valid > 0) store8(y + t * ldy + c, vec, valid, sum);
    }
}

// One warp per row r, eight columns per lane at a time; pair p = rows[r].  HBM-bound:
// reads x (for the dot product), writes dx; a token's dy comes from L2 after its first use
// (32768 rows of 2048: bfloat16 44 us, 6.4 TB/s, float32 93 us, 6.1 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) combine_backward_kernel(int64_t pairs, int top, int64_t n, const T* dy,
                                                               int64_t lddy, const T* x, int64_t ldx,
                                                               const int32_t* rows, const int32_t* slots,
                                                               const float* weights, T* dx, int64_t lddx,
                                                               float* dweights, bool vec) {
    pdl_trigger();
    pdl_wait();
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (r >= pairs) return;
    const int64_t p = rows[r];
    if (dweights && lane == 0 && slots[r] < 0) dweights[r] = 0.0f;
    const bool owned = p >= 0 && p < pairs;
    const float w = owned ? (weights ? weights[p] : 1.0f) : 0.0f;
    const T* d = dy + (owned ? p / top : 0) * lddy;
    float dot = 0.0f;
    constexpr int N = sizeof(T) / 2, U = 4 / N;
    int64_t c = 8 * lane;
    if (vec && owned && dweights) {  // U steps' loads in flight
        for (; c + 256 * (U - 1) + 8 <= n; c += 256 * U) {
            uint4 g[U][N], v[U][N];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                load_raw8(x + r * ldx + c + 256 * u, v[u]);
#pragma unroll
                for (int q = 0; q < N; ++q) g[u][q] = reinterpret_cast<const uint4*>(d + c + 256 * u)[q];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    f[k] = to_float(reinterpret_cast<const T*>(g[u])[k]);
                    dot = fmaf(f[k], to_float(reinterpret_cast<const T*>(v[u])[k]), dot);
                    f[k] *= w;
                }
                if (dx) store8(dx + r * lddx + c + 256 * u, true, 8, f);
            }
        }
    }
#pragma unroll 1
    for (; c < n; c += 256) {
        const int valid = static_cast<int>(n - c);
        float g[8] = {}, v[8] = {};
        if (owned) {
            load8(d + c, vec, valid, g);
            if (dweights) load8(x + r * ldx + c, vec, valid, v);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            dot = fmaf(g[k], v[k], dot);
            g[k] *= w;
        }
        if (dx) store8(dx + r * lddx + c, vec, valid, g);
    }
    if (dweights && owned) {
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) dweights[p] = dot;
    }
}

}  // namespace

size_t bias_part_bytes(int64_t rows, int64_t n, int groups, int num_sms) {
    const int slab = slab_rows(rows, n, num_sms);
    return static_cast<size_t>((rows + slab - 1) / slab + groups) * n * 4;
}

int dact_launches(bool with_bias) { return with_bias ? 2 : 1; }

template <typename T, int PARTS>
static cudaError_t run_dact(int64_t rows, int64_t n, const void* dy, int64_t lddy, const void* z, int64_t ldz, int act,
                            bf16* dz, int64_t lddz, int groups, const int32_t* offsets, void* dbias, float* part,
                            int num_sms, cudaStream_t st) {
    const int slab = slab_rows(rows, n, num_sms);
    const dim3 grid(static_cast<unsigned>(((rows + slab - 1) / slab) * ((n + kWidth - 1) / kWidth)));
    const bool vec = rows_aligned<T>(dy, lddy) && (act == SGEMM_ACT_NONE || rows_aligned<T>(z, ldz));
    cudaError_t e = cudaSuccess;
    if (rows > 0)
        e = launch_kernel(true, dact_kernel<T, PARTS>, grid, dim3(256), 0, st, rows, n, static_cast<const T*>(dy), lddy,
                          static_cast<const T*>(z), ldz, act, dz, lddz, groups, offsets, dbias ? part : nullptr, slab, vec);
    if (dbias && e == cudaSuccess)
        e = launch_kernel(true, dbias_kernel<T>, dim3(static_cast<unsigned>((n + 31) / 32), groups), dim3(256), 0, st,
                          rows, n, offsets, static_cast<const float*>(part), static_cast<T*>(dbias), slab);
    return e;
}

// Slabs of the gate's backward pass: as slab_rows, down to 8 rows (one per thread) while that makes
// fewer than four blocks per SM.
static int gate_slab_rows(int64_t rows, int64_t n, int num_sms) {
    const int slab = slab_rows(rows, n, num_sms);
    return slab > 32 || ((rows + 31) / 32) * ((n + kWidth - 1) / kWidth) >= int64_t(4) * num_sms ? slab : 8;
}

size_t gate_part_bytes(int64_t rows, int64_t n, int num_sms) {
    const int slab = gate_slab_rows(rows, n, num_sms);
    return static_cast<size_t>((rows + slab - 1) / slab) * 2 * n * 4;
}

template <typename T, int PARTS>
static cudaError_t run_dgate(int64_t rows, int64_t n, const void* dy, int64_t lddy, const void* z, int64_t ldz, int act,
                             bf16* dz, int64_t lddz, void* dbias, float* part, int num_sms, cudaStream_t st) {
    const int slab = gate_slab_rows(rows, n, num_sms);
    const dim3 grid(static_cast<unsigned>(((rows + slab - 1) / slab) * ((n + kWidth - 1) / kWidth)));
    const bool vec = n % 8 == 0 && rows_aligned<T>(dy, lddy) && rows_aligned<T>(z, ldz);
    cudaError_t e = cudaSuccess;
    if (rows > 0)
        e = launch_kernel(true, vec ? dgate_kernel<T, PARTS, true> : dgate_kernel<T, PARTS, false>, grid, dim3(256), 0, st,
                          rows, n, static_cast<const T*>(dy), lddy, static_cast<const T*>(z), ldz, act, dz, lddz,
                          dbias ? part : nullptr, slab);
    if (dbias && e == cudaSuccess)
        e = launch_kernel(true, dbias_kernel<T>, dim3(static_cast<unsigned>((2 * n + 31) / 32), 1), dim3(256), 0, st,
                          rows, 2 * n, static_cast<const int32_t*>(nullptr), static_cast<const float*>(part),
                          static_cast<T*>(dbias), slab);
    return e;
}

cudaError_t launch_dgate(int dtype, int64_t rows, int64_t n, const void* dy, int64_t lddy, const void* z, int64_t ldz,
                         int act, bf16* dz, int64_t lddz, void* dbias, float* part, int num_sms, cudaStream_t st) {
    return dtype == SGEMM_F32 ? run_dgate<float, 3>(rows, n, dy, lddy, z, ldz, act, dz, lddz, dbias, part, num_sms, st)
                              : run_dgate<bf16, 1>(rows, n, dy, lddy, z, ldz, act, dz, lddz, dbias, part, num_sms, st);
}

cudaError_t launch_dact(int dtype, int64_t rows, int64_t n, const void* dy, int64_t lddy, const void* z, int64_t ldz,
                        int act, bf16* dz, int64_t lddz, int groups, const int32_t* offsets, void* dbias, float* part,
                        int num_sms, cudaStream_t st) {
    return dtype == SGEMM_F32
               ? run_dact<float, 3>(rows, n, dy, lddy, z, ldz, act, dz, lddz, groups, offsets, dbias, part, num_sms, st)
               : run_dact<bf16, 1>(rows, n, dy, lddy, z, ldz, act, dz, lddz, groups, offsets, dbias, part, num_sms, st);
}

template <typename T, typename TX>
static cudaError_t run_combine(int64_t tokens, int top, int64_t n, const void* x, int64_t ldx, const int32_t* slots,
                               const float* weights, const void* residual, int64_t ldr, void* y, int64_t ldy,
                               cudaStream_t st) {
    const int64_t spans = (n + 255) / 256;
    int share = 8;  // warps per token
    while (share > 1 && share / 2 >= spans) share /= 2;
    // few tokens: more blocks to each
    const int64_t blocks = (tokens * share + 7) / 8, per_token = (spans + share - 1) / share;
    const int64_t y_blocks = blocks < 512 ? (per_token < 64 ? per_token : 64) : 1;
    const bool vec = rows_aligned<TX>(x, ldx) && rows_aligned<T>(y, ldy) &&
                     (residual == nullptr || rows_aligned<T>(residual, ldr));
    return launch_kernel(true, combine_kernel<T, TX>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(y_blocks)),
                         dim3(256), 0, st, tokens, top, n, static_cast<const TX*>(x), ldx, slots, weights,
                         static_cast<const T*>(residual), ldr, static_cast<T*>(y), ldy, vec, share);
}

cudaError_t launch_combine(int dtype, bool x_f32, int64_t tokens, int top, int64_t n, const void* x, int64_t ldx,
                           const int32_t* slots, const float* weights, const void* residual, int64_t ldr, void* y,
                           int64_t ldy, cudaStream_t st) {
    if (dtype == SGEMM_F32)
        return run_combine<float, float>(tokens, top, n, x, ldx, slots, weights, residual, ldr, y, ldy, st);
    return x_f32 ? run_combine<bf16, float>(tokens, top, n, x, ldx, slots, weights, residual, ldr, y, ldy, st)
                 : run_combine<bf16, bf16>(tokens, top, n, x, ldx, slots, weights, residual, ldr, y, ldy, st);
}

template <typename T>
static cudaError_t run_combine_backward(int64_t tokens, int top, int64_t n, const void* dy, int64_t lddy,
                                        const void* x, int64_t ldx, const int32_t* rows, const int32_t* slots,
                                        const float* weights, void* dx, int64_t lddx, float* dweights,
                                        cudaStream_t st) {
    const int64_t pairs = tokens * top;
    const bool vec = rows_aligned<T>(dy, lddy) && (dweights == nullptr || rows_aligned<T>(x, ldx)) &&
                     (dx == nullptr || rows_aligned<T>(dx, lddx));
    return launch_kernel(true, combine_backward_kernel<T>, dim3(static_cast<unsigned>((pairs + 7) / 8)), dim3(256), 0, st,
                         pairs, top, n, static_cast<const T*>(dy), lddy, static_cast<const T*>(x), ldx, rows, slots,
                         weights, static_cast<T*>(dx), lddx, dweights, vec);
}

cudaError_t launch_combine_backward(int dtype, int64_t tokens, int top, int64_t n, const void* dy, int64_t lddy,
                                    const void* x, int64_t ldx, const int32_t* rows, const int32_t* slots,
                                    const float* weights, void* dx, int64_t lddx, float* dweights, cudaStream_t st) {
    return dtype == SGEMM_F32 ? run_combine_backward<float>(tokens, top, n, dy, lddy, x, ldx, rows, slots, weights, dx,
                                                            lddx, dweights, st)
                              : run_combine_backward<bf16>(tokens, top, n, dy, lddy, x, ldx, rows, slots, weights, dx,
                                                           lddx, dweights, st);
}

}  // namespace pg
