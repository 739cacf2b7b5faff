// Rounding to e4m3 with a scale per block, shared by the kernels that do it.
#pragma once

#include <cuda_fp8.h>

#include "layers.h"

namespace pg {

constexpr float kE4m3Largest = 448.0f;

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// NaN where the block holds one, infinity where it holds one: its values are then NaN or 0.
__device__ __forceinline__ float block_scale(float largest) { return max_nan(largest / kE4m3Largest, 1.17549435e-38f); }

__device__ __forceinline__ float largest8(const float (&v)[8]) {
    float m = 0.0f;  // its sign is of no use
#pragma unroll
    for (int t = 0; t < 8; ++t) asm("max.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(m) : "f"(v[t]));
    return fabsf(m);
}

// The quotients v / scale are FP32 numbers, rounded to the nearest e4m3, ties to even.  Where nothing
// can over- or underflow on the way (plain) they are formed by Markstein's method (IBM Journal of
// Research and Development 34, 1990): with r the rounded reciprocal, q = v r, and the remainder
// v - q scale, which a fused multiply-add gives exactly, q + (v - q scale) r rounds as the quotient
// does.  (A quotient of zero takes v's sign.)
struct Divisor {
    float scale, r;
    bool plain;
};
__device__ __forceinline__ bool plain(float scale) { return scale > 8.6736174e-19f && scale < 1.1529215e18f; }  // 2^-60, 2^60
__device__ __forceinline__ Divisor divisor(float scale) { return {scale, 1.0f / scale, plain(scale)}; }
__device__ __forceinline__ uint2 round8(const float (&v)[8], const Divisor& d) {
    float2 f[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const float2 x = make_float2(v[2 * t], v[2 * t + 1]);
        const float2 a = mul2(x, both(d.r)), rest = fma2(a, both(-d.scale), x);
        const float2 y = fma2(rest, both(d.r), a);
        f[t] = make_float2(copysignf(y.x, x.x), copysignf(y.y, x.y));
    }
    if (!d.plain) {
#pragma unroll
        for (int t = 0; t < 4; ++t) f[t] = make_float2(v[2 * t] / d.scale, v[2 * t + 1] / d.scale);
    }
    uint32_t h[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) h[t] = __nv_cvt_float2_to_fp8x2(f[t], __NV_SATFINITE, __NV_E4M3);
    return make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
}

}  // namespace pg
