// Declarations shared by the layer calls' translation units: element types,
// activations, and the launchers of the kernels behind sgemm_linear,
// sgemm_route, sgemm_expert_* (not part of the ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/precision_gemm.h"
#include "internal.h"

namespace pg {

using bf16 = __nv_bfloat16;

// ---- activations -----------------------------------------------------------------
//
// Formed in FP32.  Results that are rounded to bfloat16 (FAST) take the hardware's
// exponential and reciprocal (a few 2^-22) and, for the normal distribution, one
// exponential and a polynomial: Abramowitz and Stegun, Handbook of Mathematical
// Functions, 7.1.26, erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2), t = 1 / (1 + q x),
// to 1.5e-7 -- a third of the instructions of erff, and the derivative shares its
// exponential.

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 - Phi(|z|) by the polynomial, and e = exp(-z^2 / 2).
__device__ __forceinline__ float normal_tail(float z, float& e) {
    const float t = reciprocal_approx(fmaf(0.23164189f, fabsf(z), 1.0f));  // 0.3275911 / sqrt(2)
    e = exp2_approx(-0.72134752f * z * z);                                 // log2(e) / 2
    float q = fmaf(0.5307027145f, t, -0.7265760135f);                      // the coefficients halved
    q = fmaf(q, t, 0.7107068705f);
    q = fmaf(q, t, -0.142248368f);
    q = fmaf(q, t, 0.127414796f);
    return q * t * e;
}

// 1 / (1 + exp(-z)).  In float32 as exp(z) / (1 + exp(z)) for negative z, so that no divisor passes
// 2^126, where __fdividef gives zero, and a logistic down to the subnormal floats is kept.  For
// bfloat16 it is zero from z = -87.3 on, and with it silu's values under 1e-36.
template <bool FAST>
__device__ __forceinline__ float logistic(float z) {
    if (FAST) return reciprocal_approx(1.0f + exp2_approx(-1.44269504f * z));
    const float e = expf(-fabsf(z));
    return __fdividef(z < 0.0f ? e : 1.0f, 1.0f + e);
}

// max(z, 0), NaN staying NaN
__device__ __forceinline__ float relu(float z) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(z));
    return y;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_value(float z) {
    if (ACT == SGEMM_ACT_RELU) return relu(z);
    if (ACT == SGEMM_ACT_SILU) return z * logistic<FAST>(z);
    if (ACT == SGEMM_ACT_GELU) {
        if (!FAST) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
        float e;  // z Phi(z) = max(z, 0) - |z| (1 - Phi(|z|)), the second term 0 for infinities
        const float tail = normal_tail(z, e);
        return fmaf(-fminf(fabsf(z), 3.4e38f), tail, relu(z));
    }
    // (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u))
    if (ACT == SGEMM_ACT_GELU_TANH) return z * logistic<FAST>(1.59576912160573072f * (z + 0.044715f * z * z * z));
    return z;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act_derivative(float z) {
    if (ACT == SGEMM_ACT_RELU) return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    if (ACT == SGEMM_ACT_SILU) {
        const float p = logistic<FAST>(z);
        return p * fmaf(z, 1.0f - p, 1.0f);
    }
    if (ACT == SGEMM_ACT_GELU) {
        float e, cdf;
        if (FAST) {
            const float tail = normal_tail(z, e);
            cdf = z >= 0.0f ? 1.0f - tail : tail;
        } else {
            e = expf(-0.5f * z * z);
            cdf = 0.5f * (1.0f + erff(z * 0.70710678118654752f));
        }
        return fmaf(z * 0.39894228040143268f, e, cdf);
    }
    if (ACT == SGEMM_ACT_GELU_TANH) {
        const float p = logistic<FAST>(1.59576912160573072f * (z + 0.044715f * z * z * z));
        const float q = p * (1.0f - p);  // 0 from |z| of about 10 on, where z * z may overflow
        return q > 0.0f ? fmaf(z * q, 1.59576912160573072f * (1.0f + 0.134145f * z * z), p) : p;
    }
    return 1.0f;
}

// Both at once: they share the exponential.
template <int ACT, bool FAST>
__device__ __forceinline__ void act_both(float z, float& value, float& slope) {
    if (ACT == SGEMM_ACT_SILU) {
        const float p = logistic<FAST>(z);
        value = z * p;
        slope = p * fmaf(z, 1.0f - p, 1.0f);
    } else if (ACT == SGEMM_ACT_GELU && FAST) {
        float e;
        const float tail = normal_tail(z, e);
        value = fmaf(-fminf(fabsf(z), 3.4e38f), tail, relu(z));
        slope = fmaf(z * 0.39894228040143268f, e, z >= 0.0f ? 1.0f - tail : tail);
    } else {
        value = act_value<ACT, FAST>(z);
        slope = act_derivative<ACT, FAST>(z);
    }
}

// Two values at once, their multiplies and adds in packed instructions: the activation's
// backward pass is bound by instructions as much as by memory.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

template <int ACT, bool FAST>
__device__ __forceinline__ float2 act_value2(float2 z) {
    if (FAST && (ACT == SGEMM_ACT_SILU || ACT == SGEMM_ACT_GELU_TANH)) {
        const float2 w = ACT == SGEMM_ACT_SILU ? z
                                               : mul2(both(1.595769122f), fma2(mul2(mul2(both(0.044715f), z), z), z, z));
        const float2 u = mul2(both(-1.44269504f), w);
        const float2 v = add2(make_float2(exp2_approx(u.x), exp2_approx(u.y)), both(1.0f));
        return mul2(z, make_float2(reciprocal_approx(v.x), reciprocal_approx(v.y)));
    }
    if (FAST && ACT == SGEMM_ACT_GELU) {  // as act_value and normal_tail
        const float2 a = make_float2(fabsf(z.x), fabsf(z.y)), d = fma2(both(0.23164189f), a, both(1.0f));
        const float2 t = make_float2(reciprocal_approx(d.x), reciprocal_approx(d.y));
        const float2 u = mul2(mul2(both(-0.72134752f), z), z);
        float2 q = fma2(both(0.5307027145f), t, both(-0.7265760135f));
        q = fma2(q, t, both(0.7107068705f));
        q = fma2(q, t, both(-0.142248368f));
        q = fma2(q, t, both(0.127414796f));
        const float2 tail = mul2(mul2(q, t), make_float2(exp2_approx(u.x), exp2_approx(u.y)));
        return fma2(make_float2(-fminf(a.x, 3.4e38f), -fminf(a.y, 3.4e38f)), tail, make_float2(relu(z.x), relu(z.y)));
    }
    return make_float2(act_value<ACT, FAST>(z.x), act_value<ACT, FAST>(z.y));
}

template <int ACT, bool FAST>
__device__ __forceinline__ float2 act_derivative2(float2 z) {
    if (FAST && ACT == SGEMM_ACT_SILU) {
        const float2 u = mul2(both(-1.44269504f), z);
        const float2 v = add2(make_float2(exp2_approx(u.x), exp2_approx(u.y)), both(1.0f));
        const float2 p = make_float2(reciprocal_approx(v.x), reciprocal_approx(v.y));
        return mul2(p, fma2(z, fma2(p, both(-1.0f), both(1.0f)), both(1.0f)));
    }
    if (FAST && ACT == SGEMM_ACT_GELU) {  // as normal_tail; Phi(z) = 1/2 +- (1/2 - tail), the sign z's
        const float2 d = fma2(both(0.23164189f), make_float2(fabsf(z.x), fabsf(z.y)), both(1.0f));
        const float2 t = make_float2(reciprocal_approx(d.x), reciprocal_approx(d.y));
        const float2 u = mul2(mul2(both(-0.72134752f), z), z);
        const float2 e = make_float2(exp2_approx(u.x), exp2_approx(u.y));
        float2 q = fma2(both(0.5307027145f), t, both(-0.7265760135f));
        q = fma2(q, t, both(0.7107068705f));
        q = fma2(q, t, both(-0.142248368f));
        q = fma2(q, t, both(0.127414796f));
        const float2 body = fma2(mul2(q, t), make_float2(-e.x, -e.y), both(0.5f));
        const float2 density = fma2(mul2(both(0.39894228040143268f), z), e, both(0.5f));
        return add2(density, make_float2(copysignf(body.x, z.x), copysignf(body.y, z.y)));
    }
    return make_float2(act_derivative<ACT, FAST>(z.x), act_derivative<ACT, FAST>(z.y));
}

// f(integral_constant<act>).
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
    switch (act) {
        case SGEMM_ACT_RELU: f(std::integral_constant<int, SGEMM_ACT_RELU>()); break;
        case SGEMM_ACT_SILU: f(std::integral_constant<int, SGEMM_ACT_SILU>()); break;
        case SGEMM_ACT_GELU: f(std::integral_constant<int, SGEMM_ACT_GELU>()); break;
        case SGEMM_ACT_GELU_TANH: f(std::integral_constant<int, SGEMM_ACT_GELU_TANH>()); break;
        default: f(std::integral_constant<int, SGEMM_ACT_NONE>()); break;
    }
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(bf16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ bf16 from_float<bf16>(float v) { return __float2bfloat16_rn(v); }

// x as PARTS bfloat16 values whose sum it is (pack_kernel explains the parts).
template <int PARTS>
__device__ __forceinline__ void split_bf16(float x, bf16 (&part)[PARTS]) {
    part[0] = __float2bfloat16_rn(x);
    if (PARTS == 3) {
        if (!isfinite(x)) {
            part[0] = __float2bfloat16_rn(isnan(x) ? 0.0f : copysignf(1.0f, x));
            part[1] = __float2bfloat16_rn(0.0f);
            part[2] = __float2bfloat16_rn(x);
            return;
        }
        float x0 = __bfloat162float(part[0]);
        if (isinf(x0)) {  // the rounding of a finite value overflowed: truncate
            x0 = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
            part[0] = __float2bfloat16_rn(x0);
        }
        const float r1 = x - x0;
        part[1] = __float2bfloat16_rn(r1);
        part[2] = __float2bfloat16_rn(r1 - __bfloat162float(part[1]));
    }
}

// Eight consecutive elements, `valid` of them there (the rest read as zero and are not
// written); vec: all addresses are 16-byte aligned and whole eights may be accessed.
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, int valid, float (&v)[8]) {
    if (vec && valid >= 8) {
        uint4 raw[sizeof(T) / 2];
#pragma unroll
        for (int q = 0; q < static_cast<int>(sizeof(T)) / 2; ++q) raw[q] = reinterpret_cast<const uint4*>(p)[q];
        const T* e = reinterpret_cast<const T*>(raw);
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = to_float(e[t]);
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = t < valid ? to_float(p[t]) : 0.0f;
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, bool vec, int valid, const float (&v)[8]) {
    if (vec && valid >= 8) {
        uint4 raw[sizeof(T) / 2];
        T* e = reinterpret_cast<T*>(raw);
#pragma unroll
        for (int t = 0; t < 8; ++t) e[t] = from_float<T>(v[t]);
#pragma unroll
        for (int q = 0; q < static_cast<int>(sizeof(T)) / 2; ++q) reinterpret_cast<uint4*>(p)[q] = raw[q];
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
            if (t < valid) p[t] = from_float<T>(v[t]);
    }
}
// Whether every row of a matrix can be read in aligned eights.
template <typename T>
inline bool rows_aligned(const void* p, int64_t ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * sizeof(T)) % 16 == 0;
}

__device__ __forceinline__ uint32_t pack2(float2 v) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(v.y), "f"(v.x));
    return w;
}
__device__ __forceinline__ float2 unpack2(uint32_t w) {  // a bfloat16 is the upper half of its float
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// The parts of eight values, two to a word.  Values that no part's rounding carries to infinity take packed
// arithmetic, which gives split_bf16's bits; a comparison with the largest bfloat16 tells.
template <int PARTS>
__device__ __forceinline__ void split8(const float (&v)[8], uint32_t (&part)[PARTS][4]) {
    if (PARTS == 1) {
#pragma unroll
        for (int t = 0; t < 4; ++t) part[0][t] = pack2(make_float2(v[2 * t], v[2 * t + 1]));
        return;
    }
    float m = 0.0f;  // NaN where one is; its sign is of no use
#pragma unroll
    for (int t = 0; t < 8; ++t) asm("max.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(m) : "f"(v[t]));
    if (fabsf(m) <= 3.3895314e38f) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            float2 rest = make_float2(v[2 * t], v[2 * t + 1]);
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                part[q][t] = pack2(rest);
                if (q + 1 < PARTS) rest = fma2(unpack2(part[q][t]), make_float2(-1.0f, -1.0f), rest);
            }
        }
    } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            bf16 a[PARTS], b[PARTS];
            split_bf16<PARTS>(v[2 * t], a);
            split_bf16<PARTS>(v[2 * t + 1], b);
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
                part[q][t] = __bfloat16_as_ushort(a[q]) | static_cast<uint32_t>(__bfloat16_as_ushort(b[q])) << 16;
        }
    }
}
// Eight values as the parts of a bfloat16 matrix (16-byte aligned, part_stride apart).
template <int PARTS>
__device__ __forceinline__ void store_parts8(bf16* p, int64_t part_stride, const float (&v)[8]) {
    uint32_t part[PARTS][4];
    split8<PARTS>(v, part);
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
        *reinterpret_cast<uint4*>(p + q * part_stride) = make_uint4(part[q][0], part[q][1], part[q][2], part[q][3]);
}

// The matrix row that gathered row r stands for (list[r] / top), -1 for none.
__device__ __forceinline__ int64_t gathered_row(const int32_t* list, int top, int64_t r, int64_t rows) {
    const int32_t pair = list[r];
    const int32_t row = pair / top;
    return pair >= 0 && row < rows ? row : -1;
}

// Expert e's rows [first, end) of its list, clamped to the rows there are.
__device__ __forceinline__ void expert_rows(const int32_t* offsets, int e, int rows, int& first, int& end) {
    first = min(max(offsets[e], 0), rows);
    end = min(max(offsets[e + 1], first), rows);
}

// ---- products ---------------------------------------------------------------------
//
// Every layer product has the form
//
//     out[j][i] = epilogue(sum over k of A(i, k) * B(j, k)),   i contiguous in out,
//
// per group g (an expert; one group for the dense calls):
//   forward    i = feature n, j = row,        k = feature k   A = w,  B = x
//   dx         i = feature k, j = row,        k = feature n   A = w^T, B = dz
//   dw         i = feature k, j = feature n,  k = row         A = x^T, B = dz^T
// In the first two the groups share out the rows j, in the third the rows k.
struct Operand {
    const void* ptr;
    int64_t ld;        // row stride, elements
    int64_t stride;    // between groups, elements (weights)
    bool k_contiguous; // rows run along k (else along i / j)
    const int32_t* list;  // rows gathered: row r is the matrix's row list[r] / top (null: r)
    int top;
    int64_t rows;      // stored rows of the matrix (per group for weights)
    int parts;         // 0: elements of the call's dtype; 1 or 3: bfloat16 parts of it, one after
                       // another, `stride` apart, as the tensor-core kernel reads them
    bool packed;       // all ld columns of its rows are this call's own memory
};

struct Product {
    int dtype;
    int64_t ni, nj, nk;      // extents (nj or nk: all rows of all groups)
    int groups;
    const int32_t* offsets;  // groups + 1 first rows on the device (null: one group)
    bool rows_on_k;          // dw: the groups share out k
    Operand a, b;
    // epilogue: z = sum + bias; preact = z; out = act(z) + residual
    const void* bias;        // ni per group
    int act;
    const void* residual;
    int64_t ldr;
    void* out;
    int64_t ldo;
    int64_t out_stride;      // between groups (rows_on_k)
    void* preact;
    int64_t ldz;
    bool out_f32;            // out is FP32 whatever dtype (no residual, no preact)
    // A has 2 ni rows and out = act(g) v with g of row i, v of row ni + i; bias and preact hold
    // both, the gate's first (one group, rows along k, no residual).
    bool gated;
};

// ---- launchers ----
//
// Every kernel of the layer calls waits for the kernel before it (pdl_wait) before it
// touches global memory, so each is launched as a programmatic dependent of whatever
// precedes it on the stream, the caller's kernels included, and its launch latency
// hides behind that kernel's end.
// -----------------------------------------------------------------------

// Forward products of few rows (b's rows along k, out of the call's dtype).  One pass over a
// group's weights serves up to 4 rows of bfloat16 or 16 of float32, the number chosen once per
// launch from the rows of a dense call or twice the lists' average length; a longer list takes
// further passes.
cudaError_t launch_product_rows(const Product& p, int num_sms, cudaStream_t st);

// Rows (list[r] / top of src_rows, or `groups` matrices of per_group rows, `stride`
// apart) as packed bfloat16 parts of leading dimension ldd (a multiple of 8), part
// after part: one for bfloat16, three for float32.  Columns from cols rounded up to 8 on
// are not written (no product reads them).  One launch for up to two matrices.
struct PackJob {
    const void* src;
    int64_t ld, stride, groups, per_group, cols;
    const int32_t* list;
    int top;
    int64_t src_rows;
    bf16* dst;
    int64_t ldd;
    bool vec;  // set by launch_pack
};
// Leading dimension of packed rows.  Rows that start on 128-byte lines keep each row of a
// TMA box in one line (dw of 1000 x 1500 float32 over 8192 tokens: 267 -> 186 us), at most
// an eighth more memory.
inline int64_t packed_ld(int64_t cols) {
    const int64_t unit = cols >= 512 ? 64 : 8;
    return (cols + unit - 1) / unit * unit;
}
cudaError_t launch_pack(int dtype, const PackJob* jobs, int count, int num_sms, cudaStream_t st);

// Tensor-core products: tile width, tiles (an upper bound for grouped rows), K slices,
// and the workspace of the slices' blocks and their places.
struct TcPlan {
    int bn;
    bool gather;            // listed rows of b are gathered by the kernel
    int64_t tiles, whole;  // the first `whole` tiles have one slice
    int split, split_kb;
    bool halved;            // the others are halved along j instead of cut along k
    size_t part_bytes, info_bytes;
};
TcPlan plan_tc(const Product& p, int num_sms, int force_bn, int force_split);
int launch_product_tc(const CallContext& c, const Product& p, const TcPlan& t, int parts, void* ws, cudaStream_t st,
                      int* launches);

// dz = dy * act'(z) as bfloat16 parts (one for bfloat16, three for float32, rows * lddz
// apart; may be null), and per group the column sums of dz before rounding, into dbias
// (groups x n; may be null).  part: bias_part_bytes().
size_t bias_part_bytes(int64_t rows, int64_t n, int groups, int num_sms);
cudaError_t launch_dact(int dtype, int64_t rows, int64_t n, const void* dy, int64_t lddy, const void* z, int64_t ldz,
                        int act, bf16* dz, int64_t lddz, int groups, const int32_t* offsets, void* dbias, float* part,
                        int num_sms, cudaStream_t st);
int dact_launches(bool with_bias);
// The same for out = act(g) v: z = [g v] and dz = [dy v act'(g), dy act(g)] have 2 n columns, dbias 2 n
// entries (one group).  dz null: the sums alone.
size_t gate_part_bytes(int64_t rows, int64_t n, int num_sms);
cudaError_t launch_dgate(int dtype, int64_t rows, int64_t n, const void* dy, int64_t lddy, const void* z, int64_t ldz,
                         int act, bf16* dz, int64_t lddz, void* dbias, float* part, int num_sms, cudaStream_t st);

// x_f32: the rows are FP32 whatever dtype.
cudaError_t launch_combine(int dtype, bool x_f32, int64_t tokens, int top, int64_t n, const void* x, int64_t ldx,
                           const int32_t* slots, const float* weights, const void* residual, int64_t ldr, void* y,
                           int64_t ldy, cudaStream_t st);
cudaError_t launch_combine_backward(int dtype, int64_t tokens, int top, int64_t n, const void* dy, int64_t lddy,
                                    const void* x, int64_t ldx, const int32_t* rows, const int32_t* slots,
                                    const float* weights, void* dx, int64_t lddx, float* dweights, cudaStream_t st);

// e4m3 values with a scale for each 1 x 128 (block_rows 1) or 128 x 128 of the matrix (block.cu), the
// scales s_row apart along rows and s_block along blocks of k (1 for 128 x 128).
cudaError_t launch_quantize(int dtype, int64_t rows, int64_t cols, int block_rows, const void* x, int64_t ldx, uint8_t* q,
                            int64_t ldq, float* scales, int64_t s_row, int64_t s_block, int num_sms, cudaStream_t st);
// Rows of bytes copied to 16-byte boundaries.
cudaError_t launch_copy_bytes(const uint8_t* src, int64_t ld, int64_t rows, int64_t cols, uint8_t* dst, int64_t ldd,
                              int num_sms, cudaStream_t st);
// y = act(x w^T + bias) + residual of such matrices: x with scales of 1 x 128, w of 128 x 128, rows
// at 16-byte boundaries.
struct BlockProduct {
    int dtype;  // of bias, residual and y
    int64_t t, n, k;
    const uint8_t* x;
    int64_t ldx;
    const float* x_scales;
    int64_t xs_row, xs_block;
    const uint8_t* w;
    int64_t ldw;
    const float* w_scales;
    int64_t ldws;
    const void* bias;
    int act;
    const void* residual;
    int64_t ldr;
    void* y;
    int64_t ldy;
};
struct BlockPlan {
    int bn, split, split_kb;
    size_t part_bytes;
};
BlockPlan plan_block(int64_t t, int64_t n, int64_t k, int num_sms, int force_bn, int force_split);
int launch_block(const CallContext& c, const BlockProduct& p, const BlockPlan& plan, float* part, cudaStream_t st,
                 int* launches);

// The same for few rows (block_few_rows), x of the call's type (x_scales null) or e4m3.
// Values of x up to which each thread block rounds them by itself; from there on a kernel before it does.  One row
// of 1024 / 4096 / 8192 / 16384 values by 1024 / 4096 / 4096 / 512 features: 4.9 / 8.3 / 12.0 / 16.2 us by itself,
// 6.1 / 9.2 / 11.8 / 12.0 with the kernel.
constexpr int64_t kRawValues = 4096;
bool block_few_rows(int64_t t, int64_t n, int64_t k);
cudaError_t launch_block_rows(const BlockProduct& p, int num_sms, cudaStream_t st);

// Layer norm (norm.cu).  part: norm_part_bytes(), read where dw or db is asked for.
cudaError_t launch_norm(int dtype, int64_t rows, int64_t n, const void* x, int64_t ldx, const void* w, const void* b,
                        float eps, void* y, int64_t ldy, float* mean, float* rstd, int num_sms, cudaStream_t st);
size_t norm_part_bytes(int64_t rows, int64_t n, int num_sms);
int norm_backward_launches(int64_t rows, int64_t n, bool dx, bool sums);
cudaError_t launch_norm_backward(int dtype, int64_t rows, int64_t n, const void* dy, int64_t lddy, const void* x,
                                 int64_t ldx, const void* w, const float* mean, const float* rstd,
                                 const void* residual, int64_t ldr, void* dx, int64_t lddx, void* dw, void* db,
                                 float* part, int num_sms, cudaStream_t st);

cudaError_t launch_route(int dtype, int64_t tokens, int experts, int top, const void* logits, int64_t ldl, int score,
                         const float* balance, int groups, int group_top, int renorm, float scale,
                         const uint8_t* mask, float* weights, int32_t* ids, cudaStream_t st);
cudaError_t launch_route_backward(int dtype, int64_t tokens, int experts, int top, const float* dweights,
                                  const void* logits, int64_t ldl, const int32_t* ids, int score, int renorm,
                                  float scale, void* dlogits, int64_t lddl, cudaStream_t st);
size_t plan_part_bytes(int64_t pairs, int experts);
int plan_launches(int64_t pairs);
cudaError_t launch_expert_plan(int64_t pairs, int experts, const int32_t* ids, int32_t* counts, int32_t* offsets,
                               int32_t* rows, int32_t* slots, int32_t* part, cudaStream_t st);

}  // namespace pg
