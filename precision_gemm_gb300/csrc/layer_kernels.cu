// Row-wise kernels of the layer calls: the activation's backward pass with the
// bias gradient, and the weighted sum of a token's expert rows in both directions.
#include "layers.h"

namespace pg {
namespace {

constexpr int kSlab = 64;  // rows per block of the activation's backward pass

// dz = dy * act'(z) for a slab of 64 rows x 256 columns, and the slab's column
// sums per group: a slab's rows may belong to several groups, whose sums go to
// the slots slab + g of part ((slabs + groups) x n) -- slab + g grows with every
// new slab and with every new group, so no two sums share a slot.
template <typename T, int PARTS>
__global__ void __launch_bounds__(256) dact_kernel(int64_t rows, int64_t n, const T* dy, int64_t lddy, const T* z,
                                                   int64_t ldz, int act, bf16* dz, int64_t lddz, int groups,
                                                   const int32_t* offsets, float* part) {
    const int64_t c = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x;
    if (c >= n) return;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kSlab;
    const int64_t r1 = r0 + kSlab < rows ? r0 + kSlab : rows;
    int g = 0, first = 0, end = static_cast<int>(rows);
    if (offsets) {
        do expert_rows(offsets, g, static_cast<int>(rows), first, end);
        while (end <= r0 && ++g < groups);
    }
    float sum = 0.0f;
    bool any = false;
    for (int64_t r = r0; r < r1 && g < groups; ++r) {
        while (r >= end) {
            if (any && part) part[(blockIdx.x + g) * n + c] = sum;
            any = false;
            sum = 0.0f;
            if (++g == groups) break;
            expert_rows(offsets, g, static_cast<int>(rows), first, end);
        }
        if (g == groups) break;
        float d = to_float(dy[r * lddy + c]);
        if (act != SGEMM_ACT_NONE)
            with_act(act, [&](auto a) { d *= act_derivative<decltype(a)::value, PARTS == 1>(to_float(z[r * ldz + c])); });
        if (dz) {
            bf16 q[PARTS];
            split_bf16<PARTS>(d, q);
#pragma unroll
            for (int k = 0; k < PARTS; ++k) dz[(k * rows + r) * lddz + c] = q[k];
        }
        sum += d;
        any = true;
    }
    if (any && part) part[(blockIdx.x + g) * n + c] = sum;
}

// dbias[g][c] = the sums of group g's slabs, in order.
template <typename T>
__global__ void __launch_bounds__(256) dbias_kernel(int64_t rows, int64_t n, const int32_t* offsets,
                                                    const float* part, T* dbias) {
    const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int g = blockIdx.y;
    if (c >= n) return;
    int first = 0, end = static_cast<int>(rows);
    if (offsets) expert_rows(offsets, g, static_cast<int>(rows), first, end);
    float sum = 0.0f;
    if (end > first)
        for (int s = first / kSlab; s <= (end - 1) / kSlab; ++s) sum += part[(static_cast<int64_t>(s) + g) * n + c];
    dbias[g * n + c] = from_float<T>(sum);
}

template <typename T, typename TX>
__global__ void __launch_bounds__(256) combine_kernel(int top, int64_t n, int64_t rows, const TX* x, int64_t ldx,
                                                      const int32_t* slots, const float* weights, const T* residual,
                                                      int64_t ldr, T* y, int64_t ldy) {
    const int64_t t = blockIdx.x;
    for (int64_t c = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x; c < n; c += 256 * gridDim.y) {
        float sum = 0.0f;
        for (int j = 0; j < top; ++j) {
            const int64_t s = slots[t * top + j];
            if (s < 0 || s >= rows) continue;
            const float v = to_float(x[s * ldx + c]);
            sum = weights ? fmaf(weights[t * top + j], v, sum) : sum + v;
        }
        if (residual) sum += to_float(residual[t * ldr + c]);
        y[t * ldy + c] = from_float<T>(sum);
    }
}

// One warp per row r; pair p = rows[r].
template <typename T>
__global__ void __launch_bounds__(256) combine_backward_kernel(int64_t pairs, int top, int64_t n, const T* dy,
                                                               int64_t lddy, const T* x, int64_t ldx,
                                                               const int32_t* rows, const int32_t* slots,
                                                               const float* weights, T* dx, int64_t lddx,
                                                               float* dweights) {
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (r >= pairs) return;
    const int64_t p = rows[r];
    if (dweights && lane == 0 && slots[r] < 0) dweights[r] = 0.0f;
    const bool owned = p >= 0 && p < pairs;
    const float w = owned ? (weights ? weights[p] : 1.0f) : 0.0f;
    const T* d = dy + (owned ? p / top : 0) * lddy;
    float dot = 0.0f;
    for (int64_t c = lane; c < n; c += 32) {
        const float g = owned ? to_float(d[c]) : 0.0f;
        if (dx) dx[r * lddx + c] = from_float<T>(owned ? w * g : 0.0f);
        if (dweights && owned) dot = fmaf(g, to_float(x[r * ldx + c]), dot);
    }
    if (dweights && owned) {
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane == 0) dweights[p] = dot;
    }
}

}  // namespace

size_t bias_part_bytes(int64_t rows, int64_t n, int groups) {
    return static_cast<size_t>((rows + kSlab - 1) / kSlab + groups) * n * 4;
}

int dact_launches(bool with_bias) { return with_bias ? 2 : 1; }

template <typename T, int PARTS>
static cudaError_t run_dact(int64_t rows, int64_t n, const void* dy, int64_t lddy, const void* z, int64_t ldz, int act,
                            bf16* dz, int64_t lddz, int groups, const int32_t* offsets, void* dbias, float* part,
                            cudaStream_t st) {
    const unsigned cols = static_cast<unsigned>((n + 255) / 256);
    const dim3 grid(static_cast<unsigned>((rows + kSlab - 1) / kSlab), cols);
    if (rows > 0)
        dact_kernel<T, PARTS><<<grid, 256, 0, st>>>(rows, n, static_cast<const T*>(dy), lddy,
                                                    static_cast<const T*>(z), ldz, act, dz, lddz, groups, offsets,
                                                    dbias ? part : nullptr);
    if (dbias)
        dbias_kernel<T><<<dim3(cols, groups), 256, 0, st>>>(rows, n, offsets, part, static_cast<T*>(dbias));
    return cudaGetLastError();
}

cudaError_t launch_dact(int dtype, int64_t rows, int64_t n, const void* dy, int64_t lddy, const void* z, int64_t ldz,
                        int act, bf16* dz, int64_t lddz, int groups, const int32_t* offsets, void* dbias, float* part,
                        cudaStream_t st) {
    return dtype == SGEMM_F32
               ? run_dact<float, 3>(rows, n, dy, lddy, z, ldz, act, dz, lddz, groups, offsets, dbias, part, st)
               : run_dact<bf16, 1>(rows, n, dy, lddy, z, ldz, act, dz, lddz, groups, offsets, dbias, part, st);
}

template <typename T, typename TX>
static cudaError_t run_combine(int64_t tokens, int top, int64_t n, const void* x, int64_t ldx, const int32_t* slots,
                               const float* weights, const void* residual, int64_t ldr, void* y, int64_t ldy,
                               cudaStream_t st) {
    const unsigned cols = static_cast<unsigned>(n > 8 * 256 ? 8 : (n + 255) / 256);
    combine_kernel<T, TX><<<dim3(static_cast<unsigned>(tokens), cols), 256, 0, st>>>(
        top, n, tokens * top, static_cast<const TX*>(x), ldx, slots, weights, static_cast<const T*>(residual), ldr,
        static_cast<T*>(y), ldy);
    return cudaGetLastError();
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
    combine_backward_kernel<T><<<static_cast<unsigned>((pairs + 7) / 8), 256, 0, st>>>(
        pairs, top, n, static_cast<const T*>(dy), lddy, static_cast<const T*>(x), ldx, rows, slots, weights,
        static_cast<T*>(dx), lddx, dweights);
    return cudaGetLastError();
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
