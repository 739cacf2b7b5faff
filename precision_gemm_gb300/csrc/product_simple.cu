// The layer products (layers.h, struct Product) on the CUDA cores: 64 x 64 tiles
// of out, 16-deep k steps staged in shared memory as FP32, 4 x 4 results per
// thread, every element loaded with its own bounds check.  Serves every dtype,
// orientation, stride and group layout.
#include "layers.h"
#include "ptx.cuh"

namespace pg {
namespace {

constexpr int kT = 64, kK = 16;

template <typename T>
__device__ __forceinline__ float operand_at(const Operand& o, int g, int64_t row, int64_t col) {
    return to_float(static_cast<const T*>(o.ptr)[g * o.stride + row * o.ld + col]);
}

// T: operands; TO: results.
template <typename T, typename TO>
__global__ void __launch_bounds__(256) product_simple_kernel(Product p) {
    __shared__ float sa[kK][kT + 4], sb[kK][kT + 4];
    const int rows = static_cast<int>(p.rows_on_k ? p.nk : p.nj);
    // this block's group and its tile of rows j
    int g = 0, first = 0, end = rows;
    int64_t j0;
    if (p.rows_on_k) {
        g = blockIdx.z;
        j0 = static_cast<int64_t>(blockIdx.y) * kT;
        if (p.offsets) expert_rows(p.offsets, g, rows, first, end);
    } else {
        int tile = blockIdx.y;
        for (;; ++g) {
            if (g == p.groups) return;
            if (p.offsets) expert_rows(p.offsets, g, rows, first, end);
            const int tiles = (end - first + kT - 1) / kT;
            if (tile < tiles) break;
            tile -= tiles;
        }
        j0 = first + static_cast<int64_t>(tile) * kT;
    }
    const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kT;
    const int64_t j_end = p.rows_on_k ? p.nj : end;
    const int64_t k0 = p.rows_on_k ? first : 0, k_end = p.rows_on_k ? end : p.nk;
    const int ti = threadIdx.x % 16, tj = threadIdx.x / 16;
    float acc[4][4] = {};  // [j][i]
    for (int64_t kb = k0; kb < k_end; kb += kK) {
        for (int q = threadIdx.x; q < kK * kT; q += 256) {
            // along the operand's contiguous direction
            const int ka = p.a.k_contiguous ? q % kK : q / kT, ia = p.a.k_contiguous ? q / kK : q % kT;
            const int kc = p.b.k_contiguous ? q % kK : q / kT, jb = p.b.k_contiguous ? q / kK : q % kT;
            float va = 0.0f, vb = 0.0f;
            if (kb + ka < k_end && i0 + ia < p.ni) {
                if (p.a.k_contiguous) {
                    va = operand_at<T>(p.a, g, i0 + ia, kb + ka);
                } else {
                    int64_t r = kb + ka;
                    if (p.a.list) r = p.a.list[r] / p.a.top;
                    if (r >= 0 && r < p.a.rows) va = operand_at<T>(p.a, g, r, i0 + ia);
                }
            }
            if (kb + kc < k_end && j0 + jb < j_end) {
                if (p.b.k_contiguous) {
                    int64_t r = j0 + jb;
                    if (p.b.list) r = p.b.list[r] / p.b.top;
                    if (r >= 0 && r < p.b.rows) vb = operand_at<T>(p.b, 0, r, kb + kc);
                } else {
                    vb = operand_at<T>(p.b, 0, kb + kc, j0 + jb);
                }
            }
            sa[ka][ia] = va;
            sb[kc][jb] = vb;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            float a[4], b[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                a[v] = sa[k][ti + 16 * v];
                b[v] = sb[k][tj + 16 * v];
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(b[u], a[v], acc[u][v]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t j = j0 + tj + 16 * u;
        if (j >= j_end) continue;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int64_t i = i0 + ti + 16 * v;
            if (i >= p.ni) continue;
            float z = acc[u][v];
            if (p.bias) z += to_float(static_cast<const T*>(p.bias)[g * p.ni + i]);
            if (p.preact) static_cast<T*>(p.preact)[j * p.ldz + i] = from_float<T>(z);
            float y = act_value(z, p.act);
            if (p.residual) y += to_float(static_cast<const T*>(p.residual)[j * p.ldr + i]);
            static_cast<TO*>(p.out)[(p.rows_on_k ? g * p.out_stride : 0) + j * p.ldo + i] = from_float<TO>(y);
        }
    }
}

// Rows of no expert (from offsets[groups] on) are zero.
template <typename T, typename TO>
__global__ void __launch_bounds__(256) zero_rows_kernel(Product p) {
    const int64_t used = min(max(static_cast<int64_t>(p.offsets[p.groups]), int64_t(0)), p.nj);
    for (int64_t j = used + blockIdx.x; j < p.nj; j += gridDim.x) {
        for (int64_t i = threadIdx.x; i < p.ni; i += 256) {
            static_cast<TO*>(p.out)[j * p.ldo + i] = from_float<TO>(0.0f);
            if (p.preact) static_cast<T*>(p.preact)[j * p.ldz + i] = from_float<T>(0.0f);
        }
    }
}

template <typename T, typename TO>
cudaError_t run(const Product& p, cudaStream_t st) {
    const int64_t ti = (p.ni + kT - 1) / kT;
    const int64_t tj = (p.nj + kT - 1) / kT + (p.rows_on_k || p.groups == 1 ? 0 : p.groups);
    const dim3 grid(static_cast<unsigned>(ti), static_cast<unsigned>(tj), p.rows_on_k ? p.groups : 1);
    product_simple_kernel<T, TO><<<grid, 256, 0, st>>>(p);
    if (p.offsets && !p.rows_on_k) zero_rows_kernel<T, TO><<<128, 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_product_simple(const Product& p, cudaStream_t st) {
    if (p.dtype == SGEMM_F32) return run<float, float>(p, st);
    return p.out_f32 ? run<bf16, float>(p, st) : run<bf16, bf16>(p, st);
}

}  // namespace pg
