// The forward layer products (layers.h, struct Product) for few rows: a decoding
// step's tokens, or experts with a handful of rows each.  Reading the weights once is
// all there is to do (2 flops per weight and row, a few rows), so a warp streams F
// weight rows with 16-byte loads, several steps in flight, and keeps F x M sums in
// registers for M rows of x, which come from L1.  float32 weights are used as they
// are: the tensor-core path would first write them out in bfloat16 parts (10 bytes
// per weight and 6 more to read them again).  A sum is formed by 32 lanes, each over
// every 32nd group of k, in FP32; its warps' parts are added in order.
// HBM-bound: 8192 x 8192 float32, one row, 43 us (6.2 TB/s); 4096 x 4096 bfloat16, from
// HBM, 8.1 us (4.1 TB/s, start and end of the kernel included).
#include <algorithm>

#include "layers.h"
#include "ptx.cuh"

namespace pg {
namespace {

constexpr int kWarps = 8;

struct RowsParams {
    Product p;
    int ks;      // warps that share a weight row's k, 1 to kWarps
};

// 16 bytes of a weight row: read once, so they take no place in L1, which holds x.
__device__ __forceinline__ uint4 stream16(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// A lane's 16 bytes of a step, `left` elements of the row there from p on: consecutive
// elements (VEC), or every 32nd, so that a warp's single loads fall on one line where rows
// start anywhere (4096 x 4095 float32: one row 20 -> 10 us, 16 rows 57 -> 31).  FULL: the row reaches past the step.
template <typename T, bool VEC, bool FULL>
__device__ __forceinline__ uint4 load16(const T* p, int64_t left) {
    constexpr int V = 16 / sizeof(T), apart = VEC ? 1 : 32;
    if (VEC && (FULL || left >= V)) return *reinterpret_cast<const uint4*>(p);
    uint4 raw = make_uint4(0, 0, 0, 0);
    T* e = reinterpret_cast<T*>(&raw);
#pragma unroll
    for (int t = 0; t < V; ++t)
        if (FULL || t * apart < left) e[t] = p[t * apart];
    return raw;
}

__device__ __forceinline__ void unpack(const uint4& raw, float (&v)[4]) {
    v[0] = __uint_as_float(raw.x);
    v[1] = __uint_as_float(raw.y);
    v[2] = __uint_as_float(raw.z);
    v[3] = __uint_as_float(raw.w);
}
__device__ __forceinline__ void unpack(const uint4& raw, float (&v)[8]) {
    const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) {  // a bfloat16 is the upper half of its float
        v[2 * t] = __uint_as_float(u[t] << 16);
        v[2 * t + 1] = __uint_as_float(u[t] & 0xFFFF0000u);
    }
}

// M rows of x at a time, F weight rows per warp, U steps of loads in flight (VEC: all
// rows at 16-byte boundaries), B blocks per SM.
template <typename T, bool VEC, int M, int F, int U, int B>
__global__ void __launch_bounds__(32 * kWarps, B) product_rows_kernel(const RowsParams q) {
    constexpr int V = 16 / sizeof(T);
    const Product& p = q.p;
    __shared__ float sums[kWarps][F * M];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = blockIdx.y, rows = static_cast<int>(p.nj);
    pdl_trigger();
    pdl_wait();
    if (g == p.groups) {  // the rows of no expert
        const int64_t used = min(max(p.offsets[p.groups], 0), rows);
        for (int64_t j = used + blockIdx.x; j < rows; j += gridDim.x)
            for (int64_t i = threadIdx.x; i < p.ni; i += 32 * kWarps) {
                static_cast<T*>(p.out)[j * p.ldo + i] = from_float<T>(0.0f);
                if (p.preact) static_cast<T*>(p.preact)[j * p.ldz + i] = from_float<T>(0.0f);
            }
        return;
    }
    int first = 0, end = rows;
    if (p.offsets) expert_rows(p.offsets, g, rows, first, end);
    if (first >= end) return;
    const int ks = q.ks, per_block = kWarps / ks * F;
    const int part = warp % ks;
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * per_block + warp / ks * F;
    // this warp's steps of 32 V elements
    const int64_t steps = (p.nk + 32 * V - 1) / (32 * V);
    const int64_t s0 = steps * part / ks, s1 = steps * (part + 1) / ks;
    const bool all = i0 + F <= p.ni;  // F weight rows are there
    const int64_t ldw = p.a.ld;
    const int at_lane = VEC ? lane * V : lane;
    const T* w = static_cast<const T*>(p.a.ptr) + g * p.a.stride + min(i0, p.ni - 1) * ldw + at_lane;
    for (int j0 = first; j0 < end; j0 += M) {
        const T* x = static_cast<const T*>(p.b.ptr) + at_lane;
        uint32_t row[M];  // element offsets of the rows (the launcher keeps them under 2^32)
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int64_t j = min(j0 + m, end - 1);
            // a row that the list does not name loads row 0, and its sums are dropped below
            const int64_t r = p.b.list ? max(gathered_row(p.b.list, p.b.top, j, p.b.rows), int64_t(0)) : j;
            row[m] = static_cast<uint32_t>(r * p.b.ld);
        }
        float acc[F][M] = {};
        auto add = [&](const uint4(&raw)[F], const uint4& xr, int m) {
            float xv[V];
            unpack(xr, xv);
#pragma unroll
            for (int f = 0; f < F; ++f) {
                float wv[V];
                unpack(raw[f], wv);
#pragma unroll
                for (int t = 0; t < V; ++t) acc[f][m] = fmaf(wv[t], xv[t], acc[f][m]);
            }
        };
        int64_t s = s0;
        if (all) {
            const int64_t whole = min(s1, p.nk / (32 * V));  // steps without an end of a row
            // U steps' weights are on their way at any time: a step's registers are filled again as
            // soon as it is used
            uint4 raw[U][F];
            auto fetch = [&](uint4(&to)[F], int64_t at) {
                if (at < whole) {
#pragma unroll
                    for (int f = 0; f < F; ++f) {
                        const T* from = w + f * ldw + at * 32 * V;
                        to[f] = VEC ? stream16(from) : load16<T, VEC, true>(from, 0);
                    }
                }
            };
#pragma unroll
            for (int u = 0; u < U; ++u) fetch(raw[u], s + u);
            for (; s < whole; s += U) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (s + u < whole) {
#pragma unroll
                        for (int m = 0; m < M; ++m)
                            add(raw[u], load16<T, VEC, true>(x + row[m] + (s + u) * 32 * V, 0), m);
                        fetch(raw[u], s + u + U);
                    }
                }
            }
            s = whole > s0 ? whole : s0;
        }
#pragma unroll 1
        for (; s < s1; ++s) {
            const int64_t c = s * 32 * V, left = p.nk - c - at_lane;
            uint4 raw[F];
#pragma unroll
            for (int f = 0; f < F; ++f) raw[f] = load16<T, VEC, false>(w + (i0 + f < p.ni ? f : 0) * ldw + c, left);
#pragma unroll
            for (int m = 0; m < M; ++m) add(raw, load16<T, VEC, false>(x + row[m] + c, left), m);
        }
#pragma unroll
        for (int f = 0; f < F; ++f)
#pragma unroll
            for (int m = 0; m < M; ++m) {
                for (int o = 16; o > 0; o >>= 1) acc[f][m] += __shfl_xor_sync(0xffffffffu, acc[f][m], o);
                if (lane == 0) sums[warp][f * M + m] = acc[f][m];
            }
        __syncthreads();
        for (int t = threadIdx.x; t < per_block * M; t += 32 * kWarps) {
            const int m = t / per_block, li = t % per_block;  // neighbouring threads: neighbouring features
            const int64_t i = static_cast<int64_t>(blockIdx.x) * per_block + li;
            const int64_t j = j0 + m;
            if (i < p.ni && j < end) {
                float z = 0.0f;
                for (int k = 0; k < ks; ++k) z += sums[li / F * ks + k][li % F * M + m];
                if (p.b.list && gathered_row(p.b.list, p.b.top, j, p.b.rows) < 0) z = 0.0f;  // it reads as zeros
                if (p.bias) z += to_float(static_cast<const T*>(p.bias)[g * p.ni + i]);
                if (p.preact) static_cast<T*>(p.preact)[j * p.ldz + i] = from_float<T>(z);
                float y = 0.0f;
                with_act(p.act, [&](auto a) { y = act_value<decltype(a)::value, std::is_same<T, bf16>::value>(z); });
                if (p.residual) y += to_float(static_cast<const T*>(p.residual)[j * p.ldr + i]);
                static_cast<T*>(p.out)[j * p.ldo + i] = from_float<T>(y);
            }
        }
        __syncthreads();
    }
}

template <typename T, bool VEC, int M, int F, int U, int B>
cudaError_t run(const Product& p, int num_sms, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    // Enough warps to keep HBM busy: a weight row's k is shared by up to eight while there are fewer
    // than 4 B per SM (half of those that fit) and each keeps two rounds of loads (8192 x 2048
    // float32, five rows: with at least 8 B 17.8 us, 4 B 15.8; 2048 x 8192: 17.9, 15.7, 2 B 25.7).
    const int64_t active = std::max<int64_t>(1, std::min<int64_t>(p.groups, p.nj));
    const int64_t warps = (p.ni + F - 1) / F * active;
    RowsParams q{p, 1};
    while (q.ks < kWarps && warps * q.ks * 2 < kWarps * B * num_sms && p.nk >= 2 * q.ks * 2 * U * 32 * V) q.ks *= 2;
    const int64_t per_block = kWarps / q.ks * F;
    const dim3 grid(static_cast<unsigned>((p.ni + per_block - 1) / per_block), p.groups + (p.offsets ? 1 : 0));
    return launch_kernel(true, product_rows_kernel<T, VEC, M, F, U, B>, grid, dim3(32 * kWarps), 0, st, q);
}

template <typename T, bool VEC>
cudaError_t dispatch(const Product& p, int rows, int num_sms, cudaStream_t st) {
    // Up to three rows of float32, two of bfloat16, have registers for eight weight rows at once:
    // x is read half as often (HBM to registers, 8192 x 8192 float32, one row: four weight rows of
    // four steps 49.8 us, eight of two 43.5, eight of one 43.4; 2048 x 2048: 6.8, 6.0, 5.2;
    // 4096 x 4096 bfloat16: 8.7, 8.1, 9.5).  bfloat16 loaded one by one would spill.
    constexpr bool f32 = sizeof(T) == 4;
    constexpr int F = f32 || VEC ? 8 : 4, U = f32 ? 1 : 2;
    switch (rows) {
        case 1: return run<T, VEC, 1, F, U, 2>(p, num_sms, st);
        case 2: return run<T, VEC, 2, F, U, 2>(p, num_sms, st);
        case 3: return run<T, VEC, 3, f32 ? 8 : 4, f32 ? 1 : (VEC ? 4 : 2), 2>(p, num_sms, st);
        default: break;
    }
    // more than four rows of bfloat16 are a longer list's, in further passes (few_rows)
    if constexpr (std::is_same<T, float>::value) {
        switch (rows) {
            case 4: break;
            case 5: return run<T, VEC, 5, 4, 2, 2>(p, num_sms, st);
            case 6: return run<T, VEC, 6, 4, 2, 2>(p, num_sms, st);
            case 7:
            case 8: return run<T, VEC, 8, 4, 2, 2>(p, num_sms, st);
            case 9:
            case 10:
            case 11:
            case 12: return run<T, VEC, 12, 4, 1, 2>(p, num_sms, st);
            default: return run<T, VEC, 16, 4, 1, 2>(p, num_sms, st);
        }
    }
    return run<T, VEC, 4, 4, 2, 2>(p, num_sms, st);
}

template <typename T>
cudaError_t launch(const Product& p, int rows, int num_sms, cudaStream_t st) {
    const bool vec = rows_aligned<T>(p.a.ptr, p.a.ld) && p.a.stride * sizeof(T) % 16 == 0 &&
                     rows_aligned<T>(p.b.ptr, p.b.rows == 1 ? 0 : p.b.ld);
    return vec ? dispatch<T, true>(p, rows, num_sms, st)
               : dispatch<T, false>(p, rows, num_sms, st);
}

}  // namespace

cudaError_t launch_product_rows(const Product& p, int num_sms, cudaStream_t st) {
    // Rows taken together: a dense call's; of experts twice their average, since lists differ and a
    // longer one takes another pass over its weights.
    const int64_t active = std::max<int64_t>(1, std::min<int64_t>(p.groups, p.nj));
    const int rows = static_cast<int>((p.nj + active - 1) / active) * (p.groups > 1 ? 2 : 1);
    return p.dtype == SGEMM_F32 ? launch<float>(p, rows, num_sms, st)
                                : launch<bf16>(p, rows, num_sms, st);
}

}  // namespace pg
