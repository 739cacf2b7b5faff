// C ABI of the layer calls (declared in include/precision_gemm.h): argument
// checks, workspace and launch sequences of sgemm_linear, sgemm_route and
// sgemm_expert_*.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "layers.h"

#define PG_EXPORT extern "C" __attribute__((visibility("default")))

namespace pg {
namespace {

constexpr int64_t kMaxExtent = (int64_t(1) << 31) - 1024;  // TMA coordinates (tile + box) are 32-bit
constexpr int64_t kMaxLd = int64_t(1) << 36;               // TMA strides are < 2^40 bytes

size_t region(size_t bytes) { return (bytes + 255) / 256 * 256; }

// Checks that name their argument by position and name (0 when it is fine).
int check_dtype(int dtype, int pos) {
    return dtype == SGEMM_F32 || dtype == SGEMM_BF16
               ? 0
               : call_fail(-pos, "argument %d (dtype): %d is not SGEMM_F32 or SGEMM_BF16", pos, dtype);
}
int check_extent(int64_t v, int pos, const char* name, int64_t least = 0, int64_t most = kMaxExtent) {
    return v >= least && v <= most ? 0
                                   : call_fail(-pos, "argument %d (%s): %lld out of [%lld, %lld]", pos, name,
                                               (long long)v, (long long)least, (long long)most);
}
// A matrix of `cols` columns at p (used: the call touches it), its ld at pos + 1.
int check_matrix(const void* p, bool used, int64_t cols, int64_t ld, int pos, const char* name) {
    if (used && p == nullptr) return call_fail(-pos, "argument %d (%s): null pointer", pos, name);
    if (p != nullptr && (ld < std::max<int64_t>(1, cols) || ld > kMaxLd))
        return call_fail(-(pos + 1), "argument %d (ld of %s): %lld < max(1, %lld) or too large", pos + 1, name,
                         (long long)ld, (long long)cols);
    return 0;
}
int check_pointer(const void* p, bool used, int pos, const char* name) {
    return used && p == nullptr ? call_fail(-pos, "argument %d (%s): null pointer", pos, name) : 0;
}
int check_act(int act, int pos) {
    return act >= SGEMM_ACT_NONE && act <= SGEMM_ACT_GELU_TANH
               ? 0
               : call_fail(-pos, "argument %d (act): %d is not an SGEMM_ACT_* value", pos, act);
}
int check_flag(int v, int pos, const char* name) {
    return v == 0 || v == 1 ? 0 : call_fail(-pos, "argument %d (%s): %d is not 0 or 1", pos, name, v);
}

#define PG_CHECK(call)         \
    do {                       \
        const int rc_ = call;  \
        if (rc_) return rc_;   \
    } while (0)

// tokens, top and experts of an expert call (positions pos ..)
int check_pairs(int64_t tokens, int top, int pos) {
    PG_CHECK(check_extent(tokens, pos, "tokens"));
    PG_CHECK(check_extent(top, pos + 1, "top", 1, SGEMM_MAX_TOP));
    if (tokens * top > kMaxExtent)
        return call_fail(-pos, "argument %d (tokens): %lld tokens of %d choices are more than 2^31-1024 rows", pos,
                         (long long)tokens, top);
    return 0;
}

// The workspace of a call: its launch sequence runs twice, first dry to add up what it
// needs (nothing is launched), then on the memory.
struct Arena {
    char* base = nullptr;
    size_t used = 0;
    bool counting = true;
    void* take(size_t bytes) {
        char* at = base + used;
        used += region(bytes);
        return counting ? nullptr : at;
    }
    bool dry() const { return counting; }
};

template <typename F>
int with_workspace(const CallContext& c, cudaStream_t st, F body) {
    Arena sizes;
    PG_CHECK(body(sizes));
    Arena memory;
    void* ws = nullptr;
    PG_CHECK(call_workspace(c, st, sizes.used, &ws));
    memory.base = static_cast<char*>(ws);
    memory.counting = false;
    return body(memory);
}

// Whether o's rows start at 16-byte boundaries: what wide loads, and TMA of bfloat16, need.
bool rows_on_16(int dtype, const Operand& o, int groups) {
    const int64_t unit = dtype == SGEMM_F32 ? 4 : 8;
    return (reinterpret_cast<uintptr_t>(o.ptr) & 15) == 0 && o.ld % unit == 0 && (groups == 1 || o.stride % unit == 0);
}

// o as the tensor-core kernel reads it: bfloat16 rows at 16-byte aligned addresses are
// read in place; others, and float32, are packed into bfloat16 parts (a job is added).
// Listed rows are copied together unless the kernel gathers them.
int prepare(int dtype, Operand& o, int groups, int64_t cols, int64_t listed, bool gather, Arena& a, PackJob* jobs,
            int* count) {
    if (o.parts) return 0;
    const bool in_place = dtype == SGEMM_BF16 && (o.list == nullptr || gather) && rows_on_16(dtype, o, groups);
    o.parts = dtype == SGEMM_F32 ? 3 : 1;
    if (in_place) return 0;
    const int64_t per = o.list ? listed : o.rows, ldd = packed_ld(cols);
    if (o.parts * per * groups > kMaxExtent)
        return call_fail(SGEMM_ERR_TENSOR_MAP, "a float32 operand of %lld rows has more than (2^31-1024)/3",
                         (long long)(per * groups));
    bf16* dst = static_cast<bf16*>(a.take(static_cast<size_t>(o.parts) * per * groups * ldd * 2));
    PackJob& j = jobs[(*count)++];
    j = PackJob{o.ptr, o.ld, o.stride, groups, per, cols, o.list, o.top, o.rows, dst, ldd, false};
    o.ptr = dst;
    o.ld = ldd;
    o.rows = per;
    o.stride = per * ldd;
    o.list = nullptr;
    o.packed = true;
    return 0;
}

// Whether a product runs on the kernel that streams the weights once for a few rows.
// Measured against the tensor cores (us, rows / tensor cores).
// float32, whose weights those read in parts that are written first:
//   one matrix, 8192 x 2048: 8 rows 17 / 52, 16 rows 28 / 52, 24 rows 50 / 52; 2048 x 2048:
//   16 rows 14 / 20, 24 rows 25 / 20; 4096 x 64: 4 rows 4.0 / 6.9, 16 rows 11 / 6.8;
//   60 experts of 1024 x k with uneven lists, k = 64: 1 row each 12 / 18, 4 rows 33 / 20;
//   128: 4 rows 26 / 30, 8 rows 42 / 30; 256: 8 rows 49 / 53, 16 rows 72 / 54; 512: 16 rows
//   99 / 100; 2048 (64 experts): 24 rows 350 / 372, 32 rows 437 / 387 -- every pass over a
//   list ends with its warps' sums, whatever k;
//   rows at other than 16-byte boundaries: 4096 x 4095, 16 rows 31 / 59; 64 experts of 1024 x
//   2047, 16 rows 354 / 383.
// bfloat16 at 16-byte boundaries, where L2 still holds much of the matrix:
//   4096 x 4096: 1 row 5.5 / 8.8, 2 rows 7.3 / 8.8, 4 rows 9.8 / 8.8; 2048 x 8192: 2 rows
//   7.4 / 9.5, 4 rows 10.3 / 9.5; 8192 x 8192: 1 row 27 / 26, 4 rows 32 / 26;
//   64 experts of 1024 x 2048: 8 pairs 11 / 14, 32 pairs 24 / 26, 64 pairs 38 / 38; 60 of
//   1024 x 64: 5 pairs 8.0 / 5.3; of 1024 x 256: 5 pairs 5.9 / 6.2.
// bfloat16 at others, which the tensor cores read from a copy:
//   4096 x 4095: 4 rows 13 / 27, 8 rows 23 / 28; 8192 x 8191: 4 rows 52 / 90, 8 rows 105 / 90;
//   64 experts of 1024 x 2047: 64 pairs 74 / 165, 256 pairs 142 / 180, 1024 pairs 429 / 181.
bool few_rows(const Product& p) {
    if (p.rows_on_k || !p.a.k_contiguous || p.nk == 0 || p.out_f32) return false;
    if (p.b.rows * p.b.ld >= int64_t(1) << 32) return false;  // its row offsets are 32-bit
    const int64_t lists = std::min<int64_t>(p.groups, p.nj);  // lists that have rows, at most
    const bool aligned = rows_on_16(p.dtype, p.a, p.groups);
    if (p.dtype == SGEMM_F32)
        return p.groups == 1 ? p.nj <= std::min<int64_t>(16, p.nk / 8 + 1)
                             : p.nj <= lists * std::min<int64_t>(aligned ? 24 : 16, p.nk / 32 + 1);
    if (!aligned) return p.nj <= lists * std::min<int64_t>(4, p.nk / 64 + 1);
    return p.groups == 1 ? p.nj <= 3 && p.ni * p.nk <= int64_t(1) << 25 : 2 * p.nj <= p.groups && p.nk >= 256;
}

int product(const CallContext& c, Product p, Arena& a, cudaStream_t st) {
    if (p.ni == 0 || p.nj == 0) return 0;
    int launches = 0;
    if (few_rows(p)) {
        if (a.dry()) return 0;
        const cudaError_t e = launch_product_rows(p, c.sms, st);
        if (e != cudaSuccess) return call_fail_cuda(e, "layer product of few rows");
        call_count(1);
        return 0;
    }
    const TcPlan t = plan_tc(p, c.sms, c.force_bn, c.force_split);
    if (p.nk > 0) {
        const int64_t cols_a = p.a.k_contiguous ? p.nk : p.ni, cols_b = p.b.k_contiguous ? p.nk : p.nj;
        const int64_t rows_in_lists = p.rows_on_k ? p.nk : p.nj;
        PackJob jobs[2];
        int count = 0;
        PG_CHECK(prepare(p.dtype, p.a, p.rows_on_k ? 1 : p.groups, cols_a, rows_in_lists, false, a, jobs, &count));
        PG_CHECK(prepare(p.dtype, p.b, 1, cols_b, rows_in_lists, t.gather, a, jobs, &count));
        if (count > 0 && !a.dry()) {
            const cudaError_t e = launch_pack(p.dtype, jobs, count, c.sms, st);
            if (e != cudaSuccess) return call_fail_cuda(e, "operand packing");
            ++launches;
        }
    }
    void* ws = a.take(t.part_bytes + t.info_bytes);
    if (!a.dry()) {
        PG_CHECK(launch_product_tc(c, p, t, p.dtype == SGEMM_F32 ? 3 : 1, ws, st, &launches));
        call_count(launches);
    }
    return 0;
}

Operand rows_of(const void* x, int64_t ld, int64_t rows, bool k_contiguous) {
    Operand o{};
    o.ptr = x;
    o.ld = ld;
    o.k_contiguous = k_contiguous;
    o.top = 1;
    o.rows = rows;
    return o;
}

// One description for the dense and the expert backward pass.
struct Backward {
    int dtype;
    int64_t rows, n, k;  // rows of dy
    int experts;         // 1: dense
    const int32_t *offsets, *list, *slots;
    int64_t tokens;  // gather: x has this many rows
    int top;
    bool gather;
    const void *dy, *x, *w, *z;
    int64_t lddy, ldx, ldw, stride_w, ldz;
    int act;
    void *dx, *dw, *dbias;
    int64_t lddx, lddw, stride_dw;
};

int backward_steps(const CallContext& c, const Backward& b, Arena& a, cudaStream_t st) {
    cudaError_t e;
    const bool products = (b.dx || b.dw) && b.rows > 0 && b.n > 0;
    Operand dz = rows_of(b.dy, b.lddy, b.rows, true);
    // dz = dy is read in place where the tensor cores can
    const bool own_dz = products && (b.act != SGEMM_ACT_NONE || b.dtype == SGEMM_F32 || b.lddy % 8 != 0 ||
                                     (reinterpret_cast<uintptr_t>(b.dy) & 15) != 0);
    bf16* dz_own = nullptr;
    if (own_dz) {
        dz.parts = b.dtype == SGEMM_F32 ? 3 : 1;
        dz.ld = packed_ld(b.n);
        dz.stride = b.rows * dz.ld;
        dz.packed = true;
        if (dz.parts * b.rows > kMaxExtent)
            return call_fail(SGEMM_ERR_TENSOR_MAP, "a float32 operand of %lld rows has more than (2^31-1024)/3",
                             (long long)b.rows);
        dz.ptr = dz_own = static_cast<bf16*>(a.take(static_cast<size_t>(dz.parts) * dz.stride * 2));
    }
    if (own_dz || (b.dbias && b.n > 0)) {
        float* part = b.dbias ? static_cast<float*>(a.take(bias_part_bytes(b.rows, b.n, b.experts, c.sms))) : nullptr;
        if (!a.dry()) {
            if ((e = launch_dact(b.dtype, b.rows, b.n, b.dy, b.lddy, b.z, b.ldz, b.act, dz_own, dz.ld, b.experts,
                                 b.offsets, b.dbias, part, c.sms, st)) != cudaSuccess)
                return call_fail_cuda(e, "activation backward");
            call_count(dact_launches(b.dbias != nullptr));
        }
    }
    if (b.dx) {
        const bool sum_rows = b.gather;
        const int64_t ldrow = (b.k + 3) / 4 * 4;
        float* dx_rows = sum_rows ? static_cast<float*>(a.take(static_cast<size_t>(b.rows) * ldrow * 4)) : nullptr;
        Product p{};
        p.dtype = b.dtype;
        p.ni = b.k;
        p.nj = b.rows;
        p.nk = b.n;
        p.groups = b.experts;
        p.offsets = b.offsets;
        p.a = rows_of(b.w, b.ldw, b.n, false);
        p.a.stride = b.stride_w;
        p.b = dz;
        p.out = sum_rows ? static_cast<void*>(dx_rows) : b.dx;
        p.ldo = sum_rows ? ldrow : b.lddx;
        p.out_f32 = sum_rows;
        PG_CHECK(product(c, p, a, st));
        if (sum_rows && b.tokens > 0 && b.k > 0 && !a.dry()) {
            if ((e = launch_combine(b.dtype, true, b.tokens, b.top, b.k, dx_rows, ldrow, b.slots, nullptr, nullptr, 0,
                                    b.dx, b.lddx, st)) != cudaSuccess)
                return call_fail_cuda(e, "sum of the rows' gradients");
            call_count(1);
        }
    }
    if (b.dw) {
        Product p{};
        p.dtype = b.dtype;
        p.ni = b.k;
        p.nj = b.n;
        p.nk = b.rows;
        p.groups = b.experts;
        p.offsets = b.offsets;
        p.rows_on_k = true;
        p.a = rows_of(b.x, b.ldx, b.gather ? b.tokens : b.rows, false);
        if (b.gather) {
            p.a.list = b.list;
            p.a.top = b.top;
        }
        p.b = dz;
        p.b.k_contiguous = false;
        p.out = b.dw;
        p.ldo = b.lddw;
        p.out_stride = b.stride_dw;
        PG_CHECK(product(c, p, a, st));
    }
    return 0;
}

int backward(const Backward& b, cudaStream_t st) {
    CallContext c;
    PG_CHECK(call_begin(&c));
    return with_workspace(c, st, [&](Arena& a) { return backward_steps(c, b, a, st); });
}

}  // namespace
}  // namespace pg

using namespace pg;

PG_EXPORT int sgemm_linear(int dtype, int64_t t, int64_t n, int64_t k, const void* x, int64_t ldx, const void* w,
                           int64_t ldw, const void* bias, int act, const void* residual, int64_t ldr, void* y,
                           int64_t ldy, void* preact, int64_t ldz, void* stream) {
    PG_CHECK(check_dtype(dtype, 1));
    PG_CHECK(check_extent(t, 2, "t"));
    PG_CHECK(check_extent(n, 3, "n"));
    PG_CHECK(check_extent(k, 4, "k"));
    const bool some = t > 0 && n > 0;
    PG_CHECK(check_matrix(x, some && k > 0, k, ldx, 5, "x"));
    PG_CHECK(check_matrix(w, some && k > 0, k, ldw, 7, "w"));
    PG_CHECK(check_act(act, 10));
    PG_CHECK(check_matrix(residual, false, n, ldr, 11, "residual"));
    PG_CHECK(check_matrix(y, some, n, ldy, 13, "y"));
    PG_CHECK(check_matrix(preact, false, n, ldz, 15, "preact"));
    if (!some) return 0;
    CallContext c;
    PG_CHECK(call_begin(&c));
    Product p{};
    p.dtype = dtype;
    p.ni = n;
    p.nj = t;
    p.nk = k;
    p.groups = 1;
    p.a = rows_of(w, ldw, n, true);
    p.b = rows_of(x, ldx, t, true);
    p.bias = bias;
    p.act = act;
    p.residual = residual;
    p.ldr = ldr;
    p.out = y;
    p.ldo = ldy;
    p.preact = preact;
    p.ldz = ldz;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return with_workspace(c, st, [&](Arena& a) { return product(c, p, a, st); });
}

PG_EXPORT int sgemm_linear_backward(int dtype, int64_t t, int64_t n, int64_t k, const void* dy, int64_t lddy,
                                    const void* x, int64_t ldx, const void* w, int64_t ldw, int act,
                                    const void* preact, int64_t ldz, void* dx, int64_t lddx, void* dw, int64_t lddw,
                                    void* dbias, void* stream) {
    PG_CHECK(check_dtype(dtype, 1));
    PG_CHECK(check_extent(t, 2, "t"));
    PG_CHECK(check_extent(n, 3, "n"));
    PG_CHECK(check_extent(k, 4, "k"));
    PG_CHECK(check_matrix(dy, t > 0 && n > 0 && (dx || dw || dbias), n, lddy, 5, "dy"));
    PG_CHECK(check_matrix(x, t > 0 && n > 0 && k > 0 && dw, k, ldx, 7, "x"));
    PG_CHECK(check_matrix(w, t > 0 && n > 0 && k > 0 && dx, k, ldw, 9, "w"));
    PG_CHECK(check_act(act, 11));
    PG_CHECK(check_matrix(preact, t > 0 && n > 0 && act != SGEMM_ACT_NONE && (dx || dw || dbias), n, ldz, 12, "preact"));
    PG_CHECK(check_matrix(dx, false, k, lddx, 14, "dx"));
    PG_CHECK(check_matrix(dw, false, k, lddw, 16, "dw"));
    Backward b{};
    b.dtype = dtype;
    b.rows = t;
    b.n = n;
    b.k = k;
    b.experts = 1;
    b.tokens = t;
    b.top = 1;
    b.dy = dy;
    b.lddy = lddy;
    b.x = x;
    b.ldx = ldx;
    b.w = w;
    b.ldw = ldw;
    b.act = act;
    b.z = preact;
    b.ldz = ldz;
    b.dx = dx;
    b.lddx = lddx;
    b.dw = dw;
    b.lddw = lddw;
    b.dbias = dbias;
    if (!dx && !dw && !dbias) return 0;
    return backward(b, static_cast<cudaStream_t>(stream));
}

PG_EXPORT int sgemm_route(int dtype, int64_t tokens, int experts, int top, const void* logits, int64_t ldl, int score,
                          const float* balance, int groups, int group_top, int renormalize, float scale,
                          const uint8_t* mask, float* weights, int32_t* ids, void* stream) {
    PG_CHECK(check_dtype(dtype, 1));
    PG_CHECK(check_extent(tokens, 2, "tokens"));
    PG_CHECK(check_extent(experts, 3, "experts", 1, SGEMM_MAX_EXPERTS));
    PG_CHECK(check_extent(top, 4, "top", 1, std::min(experts, SGEMM_MAX_TOP)));
    PG_CHECK(check_matrix(logits, tokens > 0, experts, ldl, 5, "logits"));
    if (score != SGEMM_SCORE_SOFTMAX && score != SGEMM_SCORE_SIGMOID)
        return call_fail(-7, "argument 7 (score): %d is not an SGEMM_SCORE_* value", score);
    if (groups < 1 || groups > 32 || experts % groups != 0)
        return call_fail(-9, "argument 9 (groups): %d is no divisor of %d experts up to 32", groups, experts);
    if (group_top < 1 || group_top > groups || top > group_top * (experts / groups))
        return call_fail(-10, "argument 10 (group_top): %d of %d groups do not hold %d experts", group_top, groups, top);
    PG_CHECK(check_flag(renormalize, 11, "renormalize"));
    if (!std::isfinite(scale)) return call_fail(-12, "argument 12 (scale): %g is not finite", scale);
    PG_CHECK(check_pointer(weights, tokens > 0, 14, "weights"));
    PG_CHECK(check_pointer(ids, tokens > 0, 15, "ids"));
    if (tokens == 0) return 0;
    CallContext c;
    PG_CHECK(call_begin(&c));
    const cudaError_t e = launch_route(dtype, tokens, experts, top, logits, ldl, score, balance, groups, group_top,
                                       renormalize, scale, mask, weights, ids, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return call_fail_cuda(e, "routing");
    call_count(1);
    return 0;
}

PG_EXPORT int sgemm_route_backward(int dtype, int64_t tokens, int experts, int top, const float* dweights,
                                   const void* logits, int64_t ldl, const int32_t* ids, int score, int renormalize,
                                   float scale, void* dlogits, int64_t lddl, void* stream) {
    PG_CHECK(check_dtype(dtype, 1));
    PG_CHECK(check_extent(tokens, 2, "tokens"));
    PG_CHECK(check_extent(experts, 3, "experts", 1, SGEMM_MAX_EXPERTS));
    PG_CHECK(check_extent(top, 4, "top", 1, std::min(experts, SGEMM_MAX_TOP)));
    PG_CHECK(check_pointer(dweights, tokens > 0, 5, "dweights"));
    PG_CHECK(check_matrix(logits, tokens > 0, experts, ldl, 6, "logits"));
    PG_CHECK(check_pointer(ids, tokens > 0, 8, "ids"));
    if (score != SGEMM_SCORE_SOFTMAX && score != SGEMM_SCORE_SIGMOID)
        return call_fail(-9, "argument 9 (score): %d is not an SGEMM_SCORE_* value", score);
    PG_CHECK(check_flag(renormalize, 10, "renormalize"));
    if (!std::isfinite(scale)) return call_fail(-11, "argument 11 (scale): %g is not finite", scale);
    PG_CHECK(check_matrix(dlogits, tokens > 0, experts, lddl, 12, "dlogits"));
    if (tokens == 0) return 0;
    CallContext c;
    PG_CHECK(call_begin(&c));
    const cudaError_t e = launch_route_backward(dtype, tokens, experts, top, dweights, logits, ldl, ids, score,
                                                renormalize, scale, dlogits, lddl, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return call_fail_cuda(e, "routing backward");
    call_count(1);
    return 0;
}

PG_EXPORT int sgemm_expert_plan(int64_t tokens, int top, int experts, const int32_t* ids, int32_t* counts,
                                int32_t* offsets, int32_t* rows, int32_t* slots, void* stream) {
    PG_CHECK(check_pairs(tokens, top, 1));
    PG_CHECK(check_extent(experts, 3, "experts", 1, SGEMM_MAX_EXPERTS));
    PG_CHECK(check_pointer(ids, tokens > 0, 4, "ids"));
    PG_CHECK(check_pointer(counts, true, 5, "counts"));
    PG_CHECK(check_pointer(offsets, true, 6, "offsets"));
    PG_CHECK(check_pointer(rows, tokens > 0, 7, "rows"));
    PG_CHECK(check_pointer(slots, tokens > 0, 8, "slots"));
    CallContext c;
    PG_CHECK(call_begin(&c));
    const int64_t pairs = tokens * top;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    void* ws = nullptr;
    PG_CHECK(call_workspace(c, st, plan_part_bytes(pairs, experts), &ws));
    const cudaError_t e = launch_expert_plan(pairs, experts, ids, counts, offsets, rows, slots,
                                             static_cast<int32_t*>(ws), st);
    if (e != cudaSuccess) return call_fail_cuda(e, "expert row lists");
    call_count(plan_launches(pairs));
    return 0;
}

// tokens, top, experts, n, k, gather: arguments 2 to 7 of the expert products
static int check_expert_sizes(int64_t tokens, int top, int experts, int64_t n, int64_t k, int gather) {
    PG_CHECK(check_pairs(tokens, top, 2));
    PG_CHECK(check_extent(experts, 4, "experts", 1, SGEMM_MAX_EXPERTS));
    PG_CHECK(check_extent(n, 5, "n"));
    PG_CHECK(check_extent(k, 6, "k"));
    return check_flag(gather, 7, "gather");
}

static int check_stride(int64_t stride, bool used, int experts, int64_t n, int64_t ld, int64_t k, int pos,
                        const char* name) {
    if (used && experts > 1 && n > 0 && (stride < (n - 1) * ld + k || stride > kMaxLd))
        return call_fail(-pos, "argument %d (%s): %lld is less than one expert's matrix or too large", pos, name,
                         (long long)stride);
    return 0;
}

PG_EXPORT int sgemm_expert_linear(int dtype, int64_t tokens, int top, int experts, int64_t n, int64_t k, int gather,
                                  const void* x, int64_t ldx, const void* w, int64_t ldw, int64_t stride_w,
                                  const void* bias, int act, const int32_t* offsets, const int32_t* rows, void* y,
                                  int64_t ldy, void* preact, int64_t ldz, void* stream) {
    PG_CHECK(check_dtype(dtype, 1));
    PG_CHECK(check_expert_sizes(tokens, top, experts, n, k, gather));
    const bool some = tokens > 0 && n > 0;
    PG_CHECK(check_matrix(x, some && k > 0, k, ldx, 8, "x"));
    PG_CHECK(check_matrix(w, some && k > 0, k, ldw, 10, "w"));
    PG_CHECK(check_stride(stride_w, w != nullptr, experts, n, ldw, k, 12, "stride_w"));
    PG_CHECK(check_act(act, 14));
    PG_CHECK(check_pointer(offsets, some, 15, "offsets"));
    PG_CHECK(check_pointer(rows, some && gather, 16, "rows"));
    PG_CHECK(check_matrix(y, some, n, ldy, 17, "y"));
    PG_CHECK(check_matrix(preact, false, n, ldz, 19, "preact"));
    if (!some) return 0;
    CallContext c;
    PG_CHECK(call_begin(&c));
    Product p{};
    p.dtype = dtype;
    p.ni = n;
    p.nj = tokens * top;
    p.nk = k;
    p.groups = experts;
    p.offsets = offsets;
    p.a = rows_of(w, ldw, n, true);
    p.a.stride = stride_w;
    p.b = rows_of(x, ldx, gather ? tokens : tokens * top, true);
    if (gather) {
        p.b.list = rows;
        p.b.top = top;
    }
    p.bias = bias;
    p.act = act;
    p.out = y;
    p.ldo = ldy;
    p.preact = preact;
    p.ldz = ldz;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return with_workspace(c, st, [&](Arena& a) { return product(c, p, a, st); });
}

PG_EXPORT int sgemm_expert_linear_backward(int dtype, int64_t tokens, int top, int experts, int64_t n, int64_t k,
                                           int gather, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                           const void* w, int64_t ldw, int64_t stride_w, int act, const void* preact,
                                           int64_t ldz, const int32_t* offsets, const int32_t* rows,
                                           const int32_t* slots, void* dx, int64_t lddx, void* dw, int64_t lddw,
                                           int64_t stride_dw, void* dbias, void* stream) {
    PG_CHECK(check_dtype(dtype, 1));
    PG_CHECK(check_expert_sizes(tokens, top, experts, n, k, gather));
    const bool any = dx || dw || dbias, some = tokens > 0 && n > 0;
    PG_CHECK(check_matrix(dy, some && any, n, lddy, 8, "dy"));
    PG_CHECK(check_matrix(x, some && k > 0 && dw, k, ldx, 10, "x"));
    PG_CHECK(check_matrix(w, some && k > 0 && dx, k, ldw, 12, "w"));
    PG_CHECK(check_stride(stride_w, w != nullptr, experts, n, ldw, k, 14, "stride_w"));
    PG_CHECK(check_act(act, 15));
    PG_CHECK(check_matrix(preact, some && any && act != SGEMM_ACT_NONE, n, ldz, 16, "preact"));
    PG_CHECK(check_pointer(offsets, any, 18, "offsets"));
    PG_CHECK(check_pointer(rows, tokens > 0 && gather && dw, 19, "rows"));
    PG_CHECK(check_pointer(slots, tokens > 0 && gather && dx, 20, "slots"));
    PG_CHECK(check_matrix(dx, false, k, lddx, 21, "dx"));
    PG_CHECK(check_matrix(dw, false, k, lddw, 23, "dw"));
    PG_CHECK(check_stride(stride_dw, dw != nullptr, experts, n, lddw, k, 25, "stride_dw"));
    if (!any) return 0;
    Backward b{};
    b.dtype = dtype;
    b.rows = tokens * top;
    b.n = n;
    b.k = k;
    b.experts = experts;
    b.offsets = offsets;
    b.list = rows;
    b.slots = slots;
    b.tokens = tokens;
    b.top = top;
    b.gather = gather != 0;
    b.dy = dy;
    b.lddy = lddy;
    b.x = x;
    b.ldx = ldx;
    b.w = w;
    b.ldw = ldw;
    b.stride_w = stride_w;
    b.act = act;
    b.z = preact;
    b.ldz = ldz;
    b.dx = dx;
    b.lddx = lddx;
    b.dw = dw;
    b.lddw = lddw;
    b.stride_dw = stride_dw;
    b.dbias = dbias;
    return backward(b, static_cast<cudaStream_t>(stream));
}

PG_EXPORT int sgemm_expert_combine(int dtype, int64_t tokens, int top, int64_t n, const void* x, int64_t ldx,
                                   const int32_t* slots, const float* weights, const void* residual, int64_t ldr,
                                   void* y, int64_t ldy, void* stream) {
    PG_CHECK(check_dtype(dtype, 1));
    PG_CHECK(check_pairs(tokens, top, 2));
    PG_CHECK(check_extent(n, 4, "n"));
    const bool some = tokens > 0 && n > 0;
    PG_CHECK(check_matrix(x, some, n, ldx, 5, "x"));
    PG_CHECK(check_pointer(slots, some, 7, "slots"));
    PG_CHECK(check_matrix(residual, false, n, ldr, 9, "residual"));
    PG_CHECK(check_matrix(y, some, n, ldy, 11, "y"));
    if (!some) return 0;
    CallContext c;
    PG_CHECK(call_begin(&c));
    const cudaError_t e = launch_combine(dtype, dtype == SGEMM_F32, tokens, top, n, x, ldx, slots, weights, residual,
                                         ldr, y, ldy, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return call_fail_cuda(e, "expert combine");
    call_count(1);
    return 0;
}

PG_EXPORT int sgemm_expert_combine_backward(int dtype, int64_t tokens, int top, int64_t n, const void* dy,
                                            int64_t lddy, const void* x, int64_t ldx, const int32_t* rows,
                                            const int32_t* slots, const float* weights, void* dx, int64_t lddx,
                                            float* dweights, void* stream) {
    PG_CHECK(check_dtype(dtype, 1));
    PG_CHECK(check_pairs(tokens, top, 2));
    PG_CHECK(check_extent(n, 4, "n"));
    const bool any = dx || dweights;
    PG_CHECK(check_matrix(dy, tokens > 0 && n > 0 && any, n, lddy, 5, "dy"));
    PG_CHECK(check_matrix(x, tokens > 0 && n > 0 && dweights, n, ldx, 7, "x"));
    PG_CHECK(check_pointer(rows, tokens > 0 && any, 9, "rows"));
    PG_CHECK(check_pointer(slots, tokens > 0 && any, 10, "slots"));
    PG_CHECK(check_matrix(dx, false, n, lddx, 12, "dx"));
    if (tokens == 0 || !any) return 0;
    CallContext c;
    PG_CHECK(call_begin(&c));
    const cudaError_t e = launch_combine_backward(dtype, tokens, top, n, dy, lddy, x, ldx, rows, slots, weights, dx,
                                                  lddx, dweights, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return call_fail_cuda(e, "expert combine backward");
    call_count(1);
    return 0;
}
