// Products with 8-bit weights (block.cu) for a few rows of x, up to sixteen: a decoding step.  Reading
// the weights once is all there is to do, so they stream into registers, 16 bytes per lane and load,
// several loads in flight, and meet x in warp-level matrix instructions (m16n8k32, e4m3, FP32 sums):
// 16 weight rows by eight rows of x take two of them per 64 k and 1 KiB of weights.
//
// The order of k inside an instruction is free as long as both operands have it, so a lane's 16
// bytes of a weight row serve as they lie in memory: of a row's 64 k, lane c of four has k 16 c to 16
// c + 15, whose words 0 and 1 are one instruction's k and words 2 and 3 the next one's.
//
// x comes into every block's shared memory, e4m3 by asynchronous copies or, for few values, rounded there
// (kRawValues), while the first weights are on their way from HBM.  Up to eight warps share a weight
// row's k; their sums are added in order.
//
// Measured with quantized x (L2 cold): 1 and 8 rows x 8192 x 4096 9.4 and 10.7 us (3.6 and 3.1 TB/s), 32768 x 4096
// 27.0 and 29.3 us (5.0 and 4.6 TB/s); the tensor-core kernel of block.cu needs 14 and 32 us.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "block.cuh"
#include "layers.h"
#include "ptx.cuh"

namespace pg {
namespace {

constexpr int kWarps = 8;
constexpr int kCols = 8;         // rows of x of a matrix instruction, its columns
constexpr int kGroup = 16;       // weight rows of a warp
constexpr int kAhead = 2;        // blocks of 128 k on their way
constexpr int kBatch = 4;        // blocks of x that a thread rounds together
constexpr size_t kMostShared = 96 * 1024;

struct RowsParams {
    BlockProduct b;
    bool raw;      // x is of the call's type, not e4m3
    bool vec;      // x in 16-byte loads (raw)
    int ks;        // warps that share a weight row's k
    int kbs;
    int x_stride;  // of the rows of x in shared memory, bytes: the banks of two rows differ
};

// 16 bytes of a weight row, which no other load reads.  (A coherent load: the block may be there while an
// earlier kernel still writes the weights, and a load that takes them for constant is not for such data.)
__device__ __forceinline__ uint4 stream16(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The first `valid` bytes of v, zeros behind them.
__device__ __forceinline__ uint4 keep_bytes(uint4 v, int valid) {
    uint32_t* w = &v.x;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int bytes = valid - 4 * t;
        w[t] = bytes >= 4 ? w[t] : (bytes <= 0 ? 0u : w[t] & ((1u << (8 * bytes)) - 1));
    }
    return v;
}

// c += a b: a 16 rows x 32 k, b 32 k x 8 columns, both e4m3.
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// C matrix instructions side by side: 8 C rows of x.
template <typename T, int C>
__global__ void __launch_bounds__(32 * kWarps, 2) block_rows_kernel(const RowsParams q) {
    extern __shared__ __align__(16) uint8_t xs[];  // x's rows in e4m3, then their scales
    __shared__ float sums[kWarps][kGroup][kCols * C + 1];
    const BlockProduct& p = q.b;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, c4 = lane % 4;
    const int t = static_cast<int>(p.t), kbs = q.kbs;
    float* x_scale = reinterpret_cast<float*>(xs + static_cast<size_t>(t) * q.x_stride);  // [row][block]
    pdl_trigger();
    pdl_wait();
    const int part = warp % q.ks;
    const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * (kWarps / q.ks) + warp / q.ks) * kGroup;
    // this warp's blocks of k, the whole ones of them up to whole
    const int kb0 = kbs * part / q.ks, kb1 = kbs * (part + 1) / q.ks;
    const int whole = min(kb1, static_cast<int>(p.k / SGEMM_BLOCK));
    const uint8_t* w0 = p.w + min(i0 + g, p.n - 1) * p.ldw + 16 * c4;
    const uint8_t* w1 = p.w + min(i0 + g + 8, p.n - 1) * p.ldw + 16 * c4;
    uint4 raw[kAhead][2][2];  // [block][half][row g or g + 8]
    auto fetch = [&](uint4(&to)[2][2], int kb) {
        if (kb < whole) {
            const int64_t at = static_cast<int64_t>(kb) * SGEMM_BLOCK;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                to[h][0] = stream16(w0 + at + 64 * h);
                to[h][1] = stream16(w1 + at + 64 * h);
            }
        }
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) fetch(raw[u], kb0 + u);

    if (q.raw) {
        // sixteen lanes to a block of 128, kBatch blocks' loads in flight
        const int l16 = threadIdx.x % 16;
        for (int r = 0; r < t; ++r) {
            for (int first = 2 * warp; first < kbs; first += 2 * kBatch * kWarps) {
                float v[kBatch][8];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int kb = first + 2 * kWarps * u + lane / 16, at = kb * SGEMM_BLOCK + 8 * l16;
                    const int valid = kb < kbs ? static_cast<int>(min(max(p.k - at, int64_t(0)), int64_t(8))) : 0;
                    load8(reinterpret_cast<const T*>(p.x) + r * p.ldx + (valid > 0 ? at : 0), q.vec, valid, v[u]);
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int kb = first + 2 * kWarps * u + lane / 16;
                    if (first + 2 * kWarps * u >= kbs) break;
                    float m = largest8(v[u]);
#pragma unroll
                    for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
                    const float scale = block_scale(m);
                    const uint2 word = round8(v[u], divisor(scale));
                    if (kb < kbs) {
                        *reinterpret_cast<uint2*>(xs + r * q.x_stride + kb * SGEMM_BLOCK + 8 * l16) = word;
                        if (l16 == 0) x_scale[r * kbs + kb] = scale;
                    }
                }
            }
        }
    } else {
        // rows start at 16-byte boundaries; zeros behind k
        for (int r = 0; r < t; ++r) {
            const uint32_t to = smem_u32(xs + r * q.x_stride), to_scale = smem_u32(x_scale + r * kbs);
            for (int at = 16 * threadIdx.x; at < kbs * SGEMM_BLOCK; at += 16 * 32 * kWarps) {
                const int valid = static_cast<int>(min(max(p.k - at, int64_t(0)), int64_t(16)));
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + at),
                             "l"(p.x + r * p.ldx + (valid > 0 ? at : 0)), "r"(valid)
                             : "memory");
            }
            for (int kb = threadIdx.x; kb < kbs; kb += 32 * kWarps)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to_scale + 4 * kb),
                             "l"(p.x_scales + r * p.xs_row + kb * p.xs_block)
                             : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    __syncthreads();

    const float* sw = p.w_scales + min(i0, p.n - 1) / SGEMM_BLOCK * p.ldws;
    const uint8_t* x_row = xs + 16 * c4;
    float acc[C][4] = {};
    auto add_block = [&](const uint4(&a)[2][2], int kb, float s) {
#pragma unroll
        for (int m = 0; m < C; ++m) {
            float c[4] = {};
            const int row = kCols * m + g;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (row < t) x = *reinterpret_cast<const uint4*>(x_row + row * q.x_stride + kb * SGEMM_BLOCK + 64 * h);
                mma_e4m3(c, a[h][0].x, a[h][1].x, a[h][0].y, a[h][1].y, x.x, x.y);
                mma_e4m3(c, a[h][0].z, a[h][1].z, a[h][0].w, a[h][1].w, x.z, x.w);
            }
            const int first = kCols * m + 2 * c4;
            const float s0 = x_scale[min(first, t - 1) * kbs + kb] * s, s1 = x_scale[min(first + 1, t - 1) * kbs + kb] * s;
            acc[m][0] = fmaf(c[0], s0, acc[m][0]);
            acc[m][1] = fmaf(c[1], s1, acc[m][1]);
            acc[m][2] = fmaf(c[2], s0, acc[m][2]);
            acc[m][3] = fmaf(c[3], s1, acc[m][3]);
        }
    };
    float next_sw = kb0 < kb1 ? sw[kb0] : 0.0f;
    for (int kb = kb0; kb < whole; kb += kAhead) {
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
            if (kb + d >= whole) break;
            const float s = next_sw;
            if (kb + d + 1 < kb1) next_sw = sw[kb + d + 1];
            add_block(raw[d], kb + d, s);
            fetch(raw[d], kb + d + kAhead);
        }
    }
    if (whole < kb1) {  // the last block, which k cuts: what lies behind it in memory is no value
        const int64_t at = static_cast<int64_t>(whole) * SGEMM_BLOCK;
        uint4 a[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int left = static_cast<int>(p.k - at) - 64 * h - 16 * c4;
            a[h][0] = a[h][1] = make_uint4(0, 0, 0, 0);
            if (left > 0) {  // (a row's last 16 bytes end inside the 16-byte block of its last one)
                a[h][0] = keep_bytes(stream16(w0 + at + 64 * h), left);
                a[h][1] = keep_bytes(stream16(w1 + at + 64 * h), left);
            }
        }
        add_block(a, whole, next_sw);
    }
#pragma unroll
    for (int m = 0; m < C; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[warp][g + 8 * (e / 2)][kCols * m + 2 * c4 + e % 2] = acc[m][e];
    __syncthreads();
    const int per_block = kWarps / q.ks * kGroup;
    for (int v = threadIdx.x; v < per_block * t; v += 32 * kWarps) {
        const int m = v / per_block, li = v - m * per_block;  // neighbouring threads: neighbouring features
        const int64_t i = static_cast<int64_t>(blockIdx.x) * per_block + li;
        if (i >= p.n) continue;
        float z = 0.0f;
        for (int k = 0; k < q.ks; ++k) z += sums[li / kGroup * q.ks + k][li % kGroup][m];
        if (p.bias) z += to_float(static_cast<const T*>(p.bias)[i]);
        float y = 0.0f;
        with_act(p.act, [&](auto a) { y = act_value<decltype(a)::value, std::is_same<T, bf16>::value>(z); });
        if (p.residual) y += to_float(static_cast<const T*>(p.residual)[m * p.ldr + i]);
        static_cast<T*>(p.y)[m * p.ldy + i] = from_float<T>(y);
    }
}

}  // namespace

// Shared memory of x's rows and scales.
static size_t rows_shared(int64_t t, int64_t k) {
    const int64_t kbs = (k + SGEMM_BLOCK - 1) / SGEMM_BLOCK;
    return static_cast<size_t>(t) * (kbs * SGEMM_BLOCK + 64 + kbs * 4);
}

// Nine to sixteen rows take two instructions side by side, where that beats the tensor-core kernel with its slices
// of k: 9 and 16 rows of 1024 x 1024 6.3 and 7.7 us (7.2 and 7.5), of 4096 x 4096 8.8 and 11.3 (11.6 and 12.0), of
// 8192 x 4096 12.6 and 14.7 (14.6 and 14.8), but of 32768 x 4096 31.6 and 35.9 (32.7 and 31.0).
bool block_few_rows(int64_t t, int64_t n, int64_t k) {
    return t <= (n * k <= int64_t(1) << 25 ? 2 * kCols : kCols) && k > 0 && rows_shared(t, k) <= kMostShared;
}

cudaError_t launch_block_rows(const BlockProduct& b, int num_sms, cudaStream_t st) {
    RowsParams q{};
    q.b = b;
    q.raw = b.x_scales == nullptr;
    q.kbs = static_cast<int>((b.k + SGEMM_BLOCK - 1) / SGEMM_BLOCK);
    q.x_stride = q.kbs * SGEMM_BLOCK + 64;
    q.vec = b.dtype == SGEMM_F32 ? rows_aligned<float>(b.x, b.t == 1 ? 0 : b.ldx) : rows_aligned<bf16>(b.x, b.t == 1 ? 0 : b.ldx);
    // a weight row's k is shared while there are fewer than sixteen warps per SM and each keeps two blocks
    const int64_t groups = (b.n + kGroup - 1) / kGroup;
    q.ks = 1;
    while (q.ks < kWarps && groups * q.ks < int64_t(8) * num_sms && q.kbs >= 2 * kAhead * q.ks) q.ks *= 2;
    const int64_t per_block = kWarps / q.ks * kGroup;
    const size_t smem = rows_shared(b.t, b.k);
    auto go = [&](auto zero, auto cols) {
        using T = decltype(zero);
        auto kern = block_rows_kernel<T, decltype(cols)::value>;
        static std::atomic<uint64_t> smem_set{0};
        const cudaError_t e = set_smem_limit_once(smem_set, reinterpret_cast<const void*>(kern), static_cast<int>(kMostShared));
        if (e != cudaSuccess) return e;
        return launch_kernel(true, kern, dim3(static_cast<unsigned>((b.n + per_block - 1) / per_block)), dim3(32 * kWarps),
                             smem, st, q);
    };
    auto with_cols = [&](auto zero) {
        return b.t <= kCols ? go(zero, std::integral_constant<int, 1>()) : go(zero, std::integral_constant<int, 2>());
    };
    return b.dtype == SGEMM_F32 ? with_cols(float()) : with_cols(bf16());
}

}  // namespace pg
