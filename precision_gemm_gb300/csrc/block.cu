// Products of 8-bit matrices: e4m3 values with a float32 scale for each block of 128.
//
//     q = e4m3(x / s),  s = max(largest |x| of the block / 448, 2^-126);
//     y[j][i] = act(sum over blocks kb of 128 k of
//                   sx[j][kb] sw[i / 128][kb] sum over k in kb of xq[j][k] wq[i][k] + bias[i]) + residual[j][i]
//
// The tensor cores sum a block's 128 products (kind::f8f6f4, FP32 accumulators in TMEM); the
// scales are any FP32 numbers, so each block's sums leave TMEM and are added in registers,
// scaled, while the next block's are formed in another buffer.  sx sw is one FP32 number: below 2^-126 it
// loses bits that the block's result need not (applied in turn there, by a path of its own beside this one,
// the two cost every call 4 to 15 %).
//
// A CTA computes 128 rows j x BN features i.  Rows of x lie along TMEM lanes: a thread has one row,
// hence one sx per block, and its warp's columns are of one 128 x 128 block of w, hence one sw: a
// block's promotion is one FMA per element, two elements to an instruction.  Warp 0 loads (TMA),
// warp 1 issues the MMAs, warp 2 multiplies the scales, several blocks ahead, into shared memory;
// warps 4 to 11 promote and finish, each its quarter of the lanes and half of the columns, whose
// sums take half of the register file (setmaxnreg).  Every CTA loads its own tiles and runs its own
// MMAs (one cta_group::2 MMA for two CTAs moves a third less through shared memory, but the two
// then wait for one another's promotion of every block, 760 to 845 cycles each).
//
// For few tiles their k is cut into slices, whose scaled sums are added in slice order by
// block_sum_kernel.
//
// Bound: what a CTA's shared memory gives its MMAs.  A block of 128 x 256 x 128 reads 48 KiB of
// operands that TMA wrote there before: 768 cycles at 128 bytes each, 0.37 us at 2.07 GHz; it takes 0.40.
// Measured with quantized x, bfloat16 results (L2 cold): 4096 x 8192 x 4096 126 us (2.2 PFLOP/s), of
// which a unit's loop takes four fifths; with bias and gelu 145, with bias, silu and residual 144 (180 while
// each lane read its own row's); 1024 x 4096 x 4096 24 us, 64 x 4096 x 4096 13 us.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "block.cuh"
#include "layers.h"
#include "ptx.cuh"

namespace pg {
namespace {

constexpr int kBlock = 128;  // values that share a scale, and bytes of a shared-memory row
constexpr int kRows = 128;   // rows of x per CTA
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kCols = 32;    // columns of a TMEM load
// Registers per thread: 168 at launch, the most that 384 threads can have; 4 warps give theirs to 8.
constexpr int kRegsFew = 56, kRegsMany = 224;
static_assert(4 * kRegsFew + 8 * kRegsMany <= 12 * 168, "the shares must be there");
constexpr int kScales = 4;      // blocks of k whose scales come together
constexpr int kScaleSlots = 2;  // such groups ready or on their way
constexpr int kBiasSlots = 3;   // units whose bias is there or in use: the scales run two groups ahead, of two units at most
constexpr int kOutBytes = 64;   // of each row of a warp's results, on their way out together
constexpr int kGroupTiles = 8;  // rasterisation: tiles of rows walked before the next tile of features

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- quantization ----------------------------------------------------------------

__device__ __forceinline__ void put8(uint8_t* q, bool vec, int valid, const uint2& w) {
    if (vec && valid >= 8) {
        *reinterpret_cast<uint2*>(q) = w;
    } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
            if (t < valid) q[t] = static_cast<uint8_t>((t < 4 ? w.x : w.y) >> (8 * (t % 4)));
    }
}

// Blocks of 1 x 128: sixteen lanes to each, R neighbouring blocks of a row with their loads in
// flight.  VEC: whole eights at 16-byte boundaries (8 in q).  HBM-bound: reads x, writes a byte per
// value.
template <typename T, int R, bool VEC>
__global__ void __launch_bounds__(256) quantize_rows_kernel(int64_t rows, int64_t cols, const T* x, int64_t ldx, uint8_t* q,
                                                            int64_t ldq, float* scales, int64_t s_row, int64_t s_block) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % 16;
    const uint32_t blocks = static_cast<uint32_t>((cols + kBlock - 1) / kBlock), per_row = (blocks + R - 1) / R;
    const int64_t group = static_cast<int64_t>(blockIdx.x) * 16 + threadIdx.x / 16;
    const int64_t r = group >> 32 ? group / per_row : static_cast<uint32_t>(group) / per_row;
    const uint32_t first = static_cast<uint32_t>(group - r * per_row) * R;
    const bool there = r < rows;
    const int64_t c0 = static_cast<int64_t>(first) * kBlock + 8 * lane;
    const T* from = x + (there ? r * ldx : 0);
    float v[R][8];
    if (VEC) {
        constexpr int N = static_cast<int>(sizeof(T)) / 2;
        uint4 raw[R][N];
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int h = 0; h < N; ++h)
                raw[k][h] = there && c0 + k * kBlock < cols ? __ldcs(reinterpret_cast<const uint4*>(from + c0 + k * kBlock) + h)
                                                            : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < R; ++k)
#pragma unroll
            for (int t = 0; t < 8; ++t) v[k][t] = to_float(reinterpret_cast<const T*>(raw[k])[t]);
    } else {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t c = c0 + k * kBlock;
            load8(from + c, false, there && c < cols ? static_cast<int>(min(cols - c, int64_t(8))) : 0, v[k]);
        }
    }
    // The blocks' largest values: halves of the lanes go on with halves of the blocks, so that a lane ends with one
    // block's (its lanes / SHARE) and forms that block's divisor alone.
    constexpr int SHARE = 16 / R;
    float m[R];
#pragma unroll
    for (int k = 0; k < R; ++k) m[k] = largest8(v[k]);
    int live = R;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
        if (live > 1) {
            live /= 2;
            const bool upper = lane & o;
#pragma unroll
            for (int k = 0; k < R / 2; ++k) {
                if (k >= live) break;
                const float keep = upper ? m[k + live] : m[k], send = upper ? m[k] : m[k + live];
                m[k] = max_nan(keep, __shfl_xor_sync(0xffffffffu, send, o));
            }
        } else {
            m[0] = max_nan(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
        }
    }
    const Divisor mine = divisor(block_scale(m[0]));
    const uint32_t block = first + lane / SHARE;
    if (there && lane % SHARE == 0 && block < blocks) scales[r * s_row + block * s_block] = mine.scale;
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const float scale = __shfl_sync(0xffffffffu, mine.scale, k * SHARE, 16), inverse = __shfl_sync(0xffffffffu, mine.r, k * SHARE, 16);
        const int64_t c = c0 + k * kBlock;
        const uint2 w = round8(v[k], Divisor{scale, inverse, plain(scale)});
        if (there && c < cols) put8(q + r * ldq + c, VEC, VEC ? 8 : static_cast<int>(min(cols - c, int64_t(8))), w);
    }
}

// Blocks of 128 x 128: a thread block to each, its values kept in registers.
template <typename T>
__global__ void __launch_bounds__(256) quantize_blocks_kernel(int64_t rows, int64_t cols, const T* x, int64_t ldx,
                                                              uint8_t* q, int64_t ldq, float* scales, int64_t lds,
                                                              bool vec_x, bool vec_q) {
    __shared__ float slots[8];
    pdl_trigger();
    pdl_wait();
    const int64_t across = (cols + kBlock - 1) / kBlock, br = blockIdx.x / across, bc = blockIdx.x - br * across;
    const int64_t c = bc * kBlock + 8 * (threadIdx.x % 16);
    const int valid = static_cast<int>(min(cols - c, int64_t(8)));
    float v[8][8], m = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int64_t r = br * kBlock + 16 * k + threadIdx.x / 16;
        load8(x + (r < rows && valid > 0 ? r * ldx + c : 0), vec_x, r < rows ? valid : 0, v[k]);
        m = max_nan(m, largest8(v[k]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (threadIdx.x % 32 == 0) slots[threadIdx.x / 32] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max_nan(m, slots[k]);
    const float scale = block_scale(m);
    if (threadIdx.x == 0) scales[br * lds + bc] = scale;
    const Divisor d = divisor(scale);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int64_t r = br * kBlock + 16 * k + threadIdx.x / 16;
        if (r < rows && valid > 0) put8(q + r * ldq + c, vec_q, valid, round8(v[k], d));
    }
}

__global__ void __launch_bounds__(256) copy_bytes_kernel(const uint8_t* src, int64_t ld, int64_t rows, int64_t cols,
                                                         uint8_t* dst, int64_t ldd) {
    pdl_trigger();
    pdl_wait();
    const int64_t words = (cols + 3) / 4, count = rows * words;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < count;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r = i / words, c = 4 * (i - r * words);
        uint32_t w = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (c + t < cols) w |= static_cast<uint32_t>(src[r * ld + c + t]) << (8 * t);
        *reinterpret_cast<uint32_t*>(dst + r * ldd + c) = w;
    }
}

// ---- product ---------------------------------------------------------------------

template <int BN>
struct Cfg {
    static constexpr int A_BYTES = kRows * kBlock;
    static constexpr int B_BYTES = BN * kBlock;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES_RAW = 192 * 1024 / STAGE_BYTES;
    static constexpr int STAGES = STAGES_RAW > 10 ? 10 : STAGES_RAW;
    static constexpr int MINE = BN / 2;                // columns of an epilogue warp: a half of the tile's
    static constexpr int BUFFERS = BN == 256 ? 2 : 4;  // of TMEM: blocks of k on their way
    static constexpr uint32_t TMEM_COLS = BUFFERS * BN;
    static constexpr int BAR_BYTES = (2 * STAGES + 2 * BUFFERS + 2 * kScaleSlots + 1) * 8 + 16;
    static constexpr int OUT_BYTES = kEpiWarps * 32 * kOutBytes;
    static constexpr int SCALE_BYTES = kScaleSlots * 2 * kRows * kScales * 4;  // of the rows, for each half of the columns
    static constexpr int BIAS_BYTES = kBiasSlots * BN * 4;
    static constexpr size_t SMEM =
        1024 + static_cast<size_t>(STAGES) * STAGE_BYTES + OUT_BYTES + SCALE_BYTES + BIAS_BYTES + BAR_BYTES;
    static_assert(kEpiWarps * MINE * 4 <= SCALE_BYTES, "a bias for each warp");
    static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "slots need 1 KiB alignment");
};

struct Params {
    int32_t t, n, kbs;
    int32_t tiles_t, tiles_n;
    float inv_split, inv_t;    // reciprocals of split and tiles_t
    int32_t split, split_kb;
    const float* x_scales;
    int64_t xs_row, xs_block;  // strides along rows and along blocks of k
    const float* w_scales;
    int64_t ldws;
    const void* bias;
    int32_t act;
    const void* residual;
    int64_t ldr;
    void* y;
    int64_t ldy;
    int32_t vec;        // y, residual and bias in 16-byte accesses
    float* part;        // slices' sums, [slice][t][ldp]
    int64_t ldp;
    uint64_t timeout_ns;
    int* status;
    int32_t debug_flags;
};

struct Rows {  // of a matrix
    void* ptr;
    int64_t ld;
};

// Results of the sums v of eight columns from i on of row j, `valid` of them there.
template <typename T, int ACT>
__device__ __forceinline__ void results(const Params& p, int64_t j, int64_t i, int valid, float (&v)[8]) {
    auto add = [&](const T* from) {
        float b[8];
        load8(from, p.vec, valid, b);
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] += b[t];
    };
    if (p.bias) add(static_cast<const T*>(p.bias) + i);
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = act_value<ACT, std::is_same<T, bf16>::value>(v[t]);
    if (p.residual) add(static_cast<const T*>(p.residual) + j * p.ldr + i);
}

template <int BN, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    block_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const Params p) {
    using C = Cfg<BN>;
    constexpr int S = C::STAGES, NB = C::BUFFERS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem_1024(smem_raw);
    float4* scale_ring = reinterpret_cast<float4*>(smem + S * C::STAGE_BYTES + C::OUT_BYTES);  // [slot][half][row]
    float* biases = reinterpret_cast<float*>(smem + S * C::STAGE_BYTES + C::OUT_BYTES + C::SCALE_BYTES);  // [slot][column]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * C::STAGE_BYTES + C::OUT_BYTES + C::SCALE_BYTES + C::BIAS_BYTES);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * S + 2 * NB + 2 * kScaleSlots + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + S);
    const uint32_t acc_full0 = smem_u32(bars + 2 * S), acc_empty0 = smem_u32(bars + 2 * S + NB);
    const uint32_t scale_full0 = smem_u32(bars + 2 * S + 2 * NB), scale_empty0 = scale_full0 + 8 * kScaleSlots;
    const uint32_t mma_done = scale_empty0 + 8 * kScaleSlots;

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // known to be uniform
    const int lane = threadIdx.x & 31;
    const int first = blockIdx.x, step = gridDim.x;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(acc_full0 + 8 * b, 1);
            mbar_init(acc_empty0 + 8 * b, kEpiWarps);
        }
        for (int b = 0; b < kScaleSlots; ++b) {
            mbar_init(scale_full0 + 8 * b, 1);
            mbar_init(scale_empty0 + 8 * b, kEpiWarps);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_holder), C::TMEM_COLS);
        tmem_relinquish();
    }
    pdl_wait();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    const int units = p.tiles_t * p.tiles_n * p.split;

    struct Unit {
        int j0, i0, slice, kb0, nkb;
    };
    // a / b by b's reciprocal, a step up or down where that is off: the compiler's division of integers
    // would take a unit's every warp 150 cycles each
    auto divide = [](int a, int b, float inv, int& rest) {
        int q = __float2int_rz(static_cast<float>(a) * inv);
        rest = a - q * b;
        while (rest < 0) --q, rest += b;
        while (rest >= b) ++q, rest -= b;
        return q;
    };
    auto unit_of = [&](int u) {
        Unit x;
        const int tile = divide(u, p.split, p.inv_split, x.slice);  // the slices of a tile are neighbours
        int tt, tn;
        if (p.tiles_t <= kGroupTiles)
            tn = divide(tile, p.tiles_t, p.inv_t, tt);
        else
            tile_coords(tile, p.tiles_t, p.tiles_n, kGroupTiles, tt, tn);
        x.j0 = tt * kRows;
        x.i0 = tn * BN;
        x.kb0 = x.slice * p.split_kb;
        x.nkb = max(min(x.kb0 + p.split_kb, p.kbs) - x.kb0, 0);
        return x;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
        if (warp == 0) {
            // ---------------- TMA loader ----------------
            if (!(p.debug_flags & 1)) {
                int it = 0, slot_i = 0;
                uint32_t phase = 1;
                bool ok = true;
                for (int u = first; u < units && ok; u += step) {
                    const Unit x = unit_of(u);
                    const int ja = __shfl_sync(0xffffffffu, x.j0, 0), ib = __shfl_sync(0xffffffffu, x.i0, 0);
                    const int kb0 = __shfl_sync(0xffffffffu, x.kb0, 0), nkb = __shfl_sync(0xffffffffu, x.nkb, 0);
                    for (int kb = 0; kb < nkb; ++kb, ++it) {
                        ok = mbar_wait_short_warp(empty0 + 8 * slot_i, phase, p.timeout_ns, abort_flag);
                        if (!ok) {
                            if (lane == 0) raise_abort(abort_flag, p.status);
                            break;
                        }
                        const uint32_t bar = full0 + 8 * slot_i;
                        if (lane == 0) mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
                        const uint32_t slot = smem_u32(smem) + slot_i * C::STAGE_BYTES;
                        const int k0 = (kb0 + kb) * kBlock;
                        tma_load_3d_warp(slot, &tmX, k0, ja, 0, bar);
                        tma_load_3d_warp(slot + C::A_BYTES, &tmW, k0, ib, 0, bar);
                        if (++slot_i == S) {
                            slot_i = 0;
                            phase ^= 1;
                        }
                    }
                }
                if (lane == 0) pdl_trigger();
                if (lane == 0) {
                    // Let every copy land before the CTA may retire.
                    for (int q = max(0, it - S); q < it; ++q)
                        mbar_wait_bounded(full0 + 8 * (q % S), (q / S) & 1, p.timeout_ns, nullptr);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            // ---------------- MMA issuer ----------------
            const uint32_t slot0 = smem_u32(smem);
            const uint64_t a_desc0 = smem_desc(slot0, 16, 1024, kSwizzle128B);
            const uint64_t b_desc0 = smem_desc(slot0 + C::A_BYTES, 16, 1024, kSwizzle128B);
            const uint32_t idesc = idesc_e4m3(kRows, BN);
            int slot_i = 0, buf = 0;
            uint32_t phase = 0, acc_phase = 1;
            bool ok = true;
            // A barrier's test takes 130 cycles to answer, a quarter of a block's time: the next block's are asked
            // for before this one's MMAs are issued.
            bool ready = false, free = false;
            auto sure = [&](bool answer, uint32_t bar, uint32_t parity) {
                return __all_sync(0xffffffffu, answer) ||
                       __all_sync(0xffffffffu, mbar_wait_short(bar, parity, p.timeout_ns, abort_flag));
            };
            for (int u = first; u < units && ok; u += step) {
                const int nkb = __shfl_sync(0xffffffffu, unit_of(u).nkb, 0);
                for (int kb = 0; kb < nkb; ++kb) {
                    ok = sure(ready, full0 + 8 * slot_i, phase) && sure(free, acc_empty0 + 8 * buf, acc_phase);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t o = static_cast<uint32_t>(slot_i * C::STAGE_BYTES) >> 4, empty = empty0 + 8 * slot_i;
                    const int b = buf;
                    if (++slot_i == S) {
                        slot_i = 0;
                        phase ^= 1;
                    }
                    if (++buf == NB) {
                        buf = 0;
                        acc_phase ^= 1;
                    }
                    ready = mbar_test(full0 + 8 * slot_i, phase);
                    free = mbar_test(acc_empty0 + 8 * buf, acc_phase);
#pragma unroll
                    for (int kk = 0; kk < kBlock / 32; ++kk)
                        mma_e4m3_warp(tmem + b * BN, a_desc0 + (o + 2 * kk), b_desc0 + (o + 2 * kk), idesc, kk > 0);
                    mma_commit_warp(acc_full0 + 8 * b);
                    mma_commit_warp(empty);
                }
            }
            if (!ok && lane == 0) raise_abort(abort_flag, p.status);
            mma_commit_warp(mma_done);  // every MMA issued here has completed
            mbar_wait_bounded(mma_done, 0, p.timeout_ns, nullptr);
            __syncwarp();
        } else if (warp == 2) {
            // ---------------- scales ----------------
            // sx sw of this CTA's rows and each half of the columns, several blocks of k ahead of their use; a unit's
            // bias comes with its first ones
            int slot = 0, bias_slot = 0;
            uint32_t phase = 1;
            bool ok = true;
            for (int u = first; u < units && ok; u += step) {
                const Unit x = unit_of(u);
                const int j0 = x.j0 + lane;
                const float *sx[4], *sw[2];
#pragma unroll
                for (int r = 0; r < 4; ++r) sx[r] = p.x_scales + min(j0 + 32 * r, p.t - 1) * p.xs_row + x.kb0 * p.xs_block;
#pragma unroll
                for (int h = 0; h < 2; ++h) sw[h] = p.w_scales + min(x.i0 + C::MINE * h, p.n - 1) / kBlock * p.ldws + x.kb0;
                for (int kb = 0; kb < x.nkb && ok; kb += kScales) {
                    float a[4][kScales], b[2][kScales];
#pragma unroll
                    for (int d = 0; d < kScales; ++d) {
                        const int at = min(kb + d, x.nkb - 1);
#pragma unroll
                        for (int r = 0; r < 4; ++r) a[r][d] = sx[r][at * p.xs_block];
#pragma unroll
                        for (int h = 0; h < 2; ++h) b[h][d] = sw[h][at];
                    }
                    ok = mbar_wait_short_warp(scale_empty0 + 8 * slot, phase, p.timeout_ns, abort_flag);
                    if (!ok) {
                        if (lane == 0) raise_abort(abort_flag, p.status);
                        break;
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            scale_ring[(2 * slot + h) * kRows + 32 * r + lane] =
                                make_float4(a[r][0] * b[h][0], a[r][1] * b[h][1], a[r][2] * b[h][2], a[r][3] * b[h][3]);
                    if (kb == 0 && p.bias && !p.part) {
#pragma unroll
                        for (int c = lane; c < BN; c += 32)
                            if (x.i0 + c < p.n) biases[bias_slot * BN + c] = to_float(static_cast<const T*>(p.bias)[x.i0 + c]);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(scale_full0 + 8 * slot);
                    if (++slot == kScaleSlots) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (++bias_slot == kBiasSlots) bias_slot = 0;
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
        // ---------------- promotion and epilogue (warps 4..11) ----------------
        const int q = warp & 3;            // TMEM lane quarter this warp may access
        const int half = (warp - 4) >> 2;  // its half of the columns
        const uint32_t base = tmem + (static_cast<uint32_t>(32 * q) << 16) + C::MINE * half;
        uint8_t* out = smem + S * C::STAGE_BYTES + (warp - 4) * (32 * kOutBytes);
        const bool one = lane == 0;
        auto free_buffer = [&](int b) {
            tc_fence_before_sync();
            __syncwarp();
            mbar_arrive_relaxed_if(one, acc_empty0 + 8 * b);
        };
        int buf = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        int slot = 0, bias_slot = 0;
        uint32_t scale_phase = 0;
        for (int u = first; u < units && ok; u += step) {
            const Unit x = unit_of(u);
            const int row0 = x.j0 + 32 * q;
            const int64_t j = row0 + lane;
            const int i0 = x.i0 + C::MINE * half;
            const bool there = row0 < p.t && i0 < p.n;  // of the warp
            if (p.residual && j < p.t && i0 < p.n) {
                // the residual comes into L2 while the MMAs run
                const T* r = static_cast<const T*>(p.residual) + j * p.ldr + i0;
                for (int c = 0; c < C::MINE && i0 + c < p.n; c += 128 / static_cast<int>(sizeof(T))) prefetch_l2(r + c);
            }
            float2 acc[C::MINE / 2];
#pragma unroll
            for (int c = 0; c < C::MINE / 2; ++c) acc[c] = make_float2(0.0f, 0.0f);
            int last = 0;  // the buffer of the last block, which the results go through
            constexpr int CHUNKS = C::MINE / kCols;
            uint32_t v[2][kCols];
            float2 scale = make_float2(0.0f, 0.0f);
            auto add_chunk = [&](int c) {
#pragma unroll
                for (int k = 0; k < kCols / 2; ++k)
                    acc[kCols / 2 * c + k] =
                        fma2(make_float2(__uint_as_float(v[c & 1][2 * k]), __uint_as_float(v[c & 1][2 * k + 1])), scale,
                             acc[kCols / 2 * c + k]);
            };
            auto wait_sums = [&]() {
                ok &= mbar_wait_short_warp(acc_full0 + 8 * buf, acc_phase, p.timeout_ns, abort_flag);
                tc_fence_after_sync();
            };
            auto first_chunks = [&]() {
                tmem_ld_32x32b_x32(base + buf * BN, v[0]);
                if (CHUNKS > 1) tmem_ld_32x32b_x32(base + buf * BN + kCols, v[1]);
            };
            auto advance = [&]() {  // to the next buffer
                last = buf;
                if (++buf == NB) {
                    buf = 0;
                    acc_phase ^= 1;
                }
            };
            // (After a wait that ran out, the loop goes on without waiting: a branch for it in here would cost
            // every block.)
            if (x.nkb > 0) {
                wait_sums();
                if (there) first_chunks();
            }
#pragma unroll 1
            for (int g = 0; g < x.nkb; g += kScales) {
                ok &= mbar_wait_short_warp(scale_full0 + 8 * slot, scale_phase, p.timeout_ns, abort_flag);
                float4 s = scale_ring[(2 * slot + half) * kRows + 32 * q + lane];
                __syncwarp();
                if (lane == 0) mbar_arrive(scale_empty0 + 8 * slot);
                if (++slot == kScaleSlots) {
                    slot = 0;
                    scale_phase ^= 1;
                }
                const int blocks = min(x.nkb - g, kScales);
                if (!there) {
                    for (int r = 0; r < blocks; ++r) {
                        advance();
                        if (g + r + 1 < x.nkb) {
                            free_buffer(last);
                            wait_sums();
                        }
                    }
                    continue;
                }
                // A block's sums come in chunks of 32 columns, two on their way at a time; while the last of them
                // is added, the next block's barrier is tested, which takes 130 cycles to answer.
#pragma unroll 1
                for (int r = 0; r < blocks; ++r) {
                    const bool more = g + r + 1 < x.nkb;
                    const uint32_t at = base + buf * BN;
                    scale = both(s.x);
                    s = make_float4(s.y, s.z, s.w, 0.0f);
                    advance();
                    tmem_wait_ld(v[0]);
                    if (CHUNKS > 1) tmem_wait_ld(v[1]);
#pragma unroll
                    for (int c = 0; c + 2 < CHUNKS; ++c) {
                        add_chunk(c);
                        tmem_ld_32x32b_x32(at + kCols * (c + 2), v[c & 1]);
                    }
                    if (CHUNKS > 2) {
                        tmem_wait_ld(v[0]);
                        tmem_wait_ld(v[1]);
                    }
                    if (more) free_buffer(last);
                    if (CHUNKS > 1) add_chunk(CHUNKS - 2);
                    bool ready = true;
                    if (more) ready = mbar_try_wait(acc_full0 + 8 * buf, acc_phase);
                    add_chunk(CHUNKS - 1);
                    if (more) {
                        if (!__all_sync(0xffffffffu, ready))
                            ok &= mbar_wait_short_warp(acc_full0 + 8 * buf, acc_phase, p.timeout_ns, abort_flag);
                        tc_fence_after_sync();
                        first_chunks();
                    }
                }
            }
            if (!ok) {
                if (lane == 0) raise_abort(abort_flag, p.status);
                break;
            }
            // The results go back to the warp's own columns of the last buffer and from there, 64 bytes of
            // a row at a time, through the epilogue: a loop, where registers would want it written out.
            const uint32_t at = base + last * BN;
            if (there) {
#pragma unroll
                for (int c = 0; c < C::MINE / kCols; ++c) {
                    uint32_t v[kCols];
#pragma unroll
                    for (int k = 0; k < kCols / 2; ++k) {
                        v[2 * k] = __float_as_uint(acc[kCols / 2 * c + k].x);
                        v[2 * k + 1] = __float_as_uint(acc[kCols / 2 * c + k].y);
                    }
                    __syncwarp();
                    tmem_st_32x32b_x32(at + kCols * c, v);
                }
                tmem_wait_st();
                // (without blocks of k no scales came, and no bias with them: their place is free)
                float* const bias = x.nkb > 0 ? biases + bias_slot * BN + C::MINE * half
                                              : reinterpret_cast<float*>(scale_ring) + C::MINE * (warp - 4);
                if (x.nkb == 0 && p.bias)
                    for (int c = lane; c < C::MINE && i0 + c < p.n; c += 32)
                        bias[c] = to_float(static_cast<const T*>(p.bias)[i0 + c]);
                __syncwarp();
                // The columns as elements TO, 64 bytes of 32 rows at a time.  They change places in shared memory
                // (16-byte words, swizzled so that eight rows' words fall on all banks), so that four lanes write
                // a row's 64 bytes together; the residual comes the same way round before.
                auto emit = [&](auto element, Rows rows_of, bool vec, const void* residual, auto value) {
                    using TO = decltype(element);
                    constexpr int SPAN = kOutBytes / static_cast<int>(sizeof(TO)), N = static_cast<int>(sizeof(TO)) / 2;
                    const int64_t row = row0 + lane / 4;
                    const int i4 = i0 + (lane & 3) * (16 / static_cast<int>(sizeof(TO))), rows_left = p.t - row0 - lane / 4;
                    TO* const shared_out = static_cast<TO*>(rows_of.ptr) + row * rows_of.ld + i4;
                    auto word = [&](int r, int q) {  // 16-byte word q of row r
                        return reinterpret_cast<uint4*>(out + kOutBytes * r + 16 * (q ^ ((r >> 1) & 3)));
                    };
                    uint4 rest[4] = {};  // (left undefined where there is no residual, they cost 336 bytes of spills)
                    auto fetch = [&](int c) {
                        if (!residual || !vec || c >= C::MINE || p.n - i0 - c < SPAN) return;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (8 * r < rows_left)
                                rest[r] = *reinterpret_cast<const uint4*>(static_cast<const TO*>(residual) + (row + 8 * r) * p.ldr + i4 + c);
                    };
                    fetch(0);
#pragma unroll 1
                    for (int c = 0; c < C::MINE && i0 + c < p.n; c += SPAN) {
                        uint32_t v[SPAN];
                        __syncwarp();
                        if constexpr (SPAN == 32)
                            tmem_ld_32x32b_x32(at + c, v);
                        else
                            tmem_ld_32x32b_x16(at + c, v);
                        const bool whole = vec && p.n - i0 - c >= SPAN;
                        if (whole && residual) {
#pragma unroll
                            for (int r = 0; r < 4; ++r) *word(8 * r + lane / 4, lane & 3) = rest[r];
                            __syncwarp();
                            fetch(c + SPAN);
                        }
                        tmem_wait_ld(v);
                        float f[SPAN];
#pragma unroll
                        for (int k = 0; k < SPAN; ++k) f[k] = __uint_as_float(v[k]);
                        value(c, f);
                        if (whole) {
                            if (residual) {
#pragma unroll
                                for (int h = 0; h < SPAN; h += 8) {
                                    TO e[8];
#pragma unroll
                                    for (int k = 0; k < N; ++k) reinterpret_cast<uint4*>(e)[k] = *word(lane, h / 8 * N + k);
#pragma unroll
                                    for (int k = 0; k < 8; ++k) f[h + k] += to_float(e[k]);
                                }
                            }
#pragma unroll
                            for (int h = 0; h < SPAN; h += 8) {
                                TO e[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k) e[k] = from_float<TO>(f[h + k]);
#pragma unroll
                                for (int k = 0; k < N; ++k) *word(lane, h / 8 * N + k) = reinterpret_cast<const uint4*>(e)[k];
                            }
                            __syncwarp();
                            uint4 w[4];
#pragma unroll
                            for (int r = 0; r < 4; ++r) w[r] = *word(8 * r + lane / 4, lane & 3);
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (8 * r < rows_left) *reinterpret_cast<uint4*>(shared_out + c + 8 * r * rows_of.ld) = w[r];
                        } else if (j < p.t) {
                            TO* const mine = static_cast<TO*>(rows_of.ptr) + j * rows_of.ld + i0 + c;
#pragma unroll
                            for (int k = 0; k < SPAN; ++k)
                                if (i0 + c + k < p.n) {
                                    if (residual) f[k] += to_float(static_cast<const TO*>(residual)[j * p.ldr + i0 + c + k]);
                                    mine[k] = from_float<TO>(f[k]);
                                }
                        }
                    }
                };
                if (p.part)
                    emit(float(), {p.part + static_cast<int64_t>(x.slice) * p.t * p.ldp, p.ldp}, true, nullptr, [](int, auto&) {});
                else
                    with_act(p.act, [&](auto act) {
                        emit(T(), {p.y, p.ldy}, p.vec != 0, p.residual, [&](int c, auto& f) {
                            constexpr int SPAN = sizeof(f) / sizeof(float);
                            if (p.bias) {
#pragma unroll
                                for (int k = 0; k < SPAN; k += 4) {
                                    const float4 b = *reinterpret_cast<const float4*>(bias + c + k);
                                    f[k] += b.x, f[k + 1] += b.y, f[k + 2] += b.z, f[k + 3] += b.w;
                                }
                            }
#pragma unroll
                            for (int k = 0; k < SPAN; k += 2) {
                                const float2 y = act_value2<decltype(act)::value, std::is_same<T, bf16>::value>(make_float2(f[k], f[k + 1]));
                                f[k] = y.x, f[k + 1] = y.y;
                            }
                        });
                    });
            }
            if (x.nkb > 0) free_buffer(last);
            if (++bias_slot == kBiasSlots) bias_slot = 0;
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

// The slices' sums of eight columns, added in slice order, and the epilogue.
template <typename T>
__global__ void __launch_bounds__(256) block_sum_kernel(const Params p) {
    pdl_trigger();
    pdl_wait();
    const int64_t eights = p.ldp / 8, item = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t j = item / eights, i = 8 * (item - j * eights);
    if (j >= p.t) return;
    const float* src = p.part + j * p.ldp + i;
    float v[8] = {};
#pragma unroll 8
    for (int s = 0; s < p.split; ++s, src += p.t * p.ldp) {
        const float4 a = __ldcg(reinterpret_cast<const float4*>(src)), b = __ldcg(reinterpret_cast<const float4*>(src) + 1);
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
    }
    const int valid = static_cast<int>(min(p.n - i, int64_t(8)));
    with_act(p.act, [&](auto act) { results<T, decltype(act)::value>(p, j, i, valid, v); });
    store8(static_cast<T*>(p.y) + j * p.ldy + i, p.vec, valid, v);
}

template <int BN, typename T>
cudaError_t run(const CUtensorMap (&m)[2], const Params& p, int num_sms, cudaStream_t st) {
    using C = Cfg<BN>;
    auto kern = block_kernel<BN, T>;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = set_smem_limit_once(smem_set, reinterpret_cast<const void*>(kern), static_cast<int>(C::SMEM));
    if (e != cudaSuccess) return e;
    const int64_t units = static_cast<int64_t>(p.tiles_t) * p.tiles_n * p.split;
    return launch_kernel(true, kern, dim3(static_cast<unsigned>(std::min<int64_t>(units, num_sms))), dim3(kThreads),
                         C::SMEM, st, m[0], m[1], p);
}

}  // namespace

cudaError_t launch_quantize(int dtype, int64_t rows, int64_t cols, int block_rows, const void* x, int64_t ldx, uint8_t* q,
                            int64_t ldq, float* scales, int64_t s_row, int64_t s_block, int num_sms, cudaStream_t st) {
    const bool vec_q = (reinterpret_cast<uintptr_t>(q) & 7) == 0 && ldq % 8 == 0;
    auto go = [&](auto zero) {
        using T = decltype(zero);
        const bool vec_x = rows_aligned<T>(x, ldx);
        const int64_t across = cdiv(cols, kBlock);
        if (block_rows == 1) {
            const bool vec = vec_x && vec_q && cols % 8 == 0;
            // several blocks' loads per thread once that leaves each SM its threads
            constexpr int R = 8 / static_cast<int>(sizeof(T));
            const bool many = rows * across >= int64_t(R * 128) * num_sms;
            auto kern = many ? (vec ? quantize_rows_kernel<T, R, true> : quantize_rows_kernel<T, R, false>)
                             : (vec ? quantize_rows_kernel<T, 1, true> : quantize_rows_kernel<T, 1, false>);
            return launch_kernel(true, kern, dim3(static_cast<unsigned>(cdiv(rows * cdiv(across, many ? R : 1), 16))), dim3(256),
                                 0, st, rows, cols, static_cast<const T*>(x), ldx, q, ldq, scales, s_row, s_block);
        }
        return launch_kernel(true, quantize_blocks_kernel<T>, dim3(static_cast<unsigned>(cdiv(rows, kBlock) * across)),
                             dim3(256), 0, st, rows, cols, static_cast<const T*>(x), ldx, q, ldq, scales, s_row, vec_x, vec_q);
    };
    return dtype == SGEMM_F32 ? go(float()) : go(bf16());
}

cudaError_t launch_copy_bytes(const uint8_t* src, int64_t ld, int64_t rows, int64_t cols, uint8_t* dst, int64_t ldd,
                              int num_sms, cudaStream_t st) {
    const int64_t blocks = std::min<int64_t>(cdiv(rows * cdiv(cols, 4), 256), int64_t(16) * num_sms);
    return launch_kernel(true, copy_bytes_kernel, dim3(static_cast<unsigned>(std::max<int64_t>(blocks, 1))), dim3(256), 0, st,
                         src, ld, rows, cols, dst, ldd);
}

BlockPlan plan_block(int64_t t, int64_t n, int64_t k, int num_sms, int force_bn, int force_split) {
    const int at_once = std::max(num_sms, 1);
    const int64_t kb = cdiv(k, kBlock);
    BlockPlan best{};
    double best_us = 0.0;
    for (int bn : {256, 128, 64}) {
        if (force_bn && force_bn <= 256 && bn != force_bn) continue;
        // microseconds of a block of k and of a tile's ends, measured at 1024 x 4096 by k of 2048 to 14336
        const double step = bn == 256 ? 0.40 : (bn == 128 ? 0.22 : 0.18), end = bn == 256 ? 3.2 : (bn == 128 ? 1.9 : 1.5);
        const int64_t tiles = cdiv(t, kRows) * cdiv(n, bn);
        const int64_t forced = std::min<int64_t>(force_split, std::max<int64_t>(kb, 1));
        const int64_t most = force_split ? forced : std::max<int64_t>(std::min<int64_t>(kb, 3 * at_once / tiles), 1);
        for (int64_t want = force_split ? forced : 1; want <= most; ++want) {
            const int64_t split_kb = std::max<int64_t>(cdiv(kb, want), 1), split = std::max<int64_t>(cdiv(kb, split_kb), 1);
            const double us = static_cast<double>(cdiv(tiles * split, at_once)) * (split_kb * step + end) +
                              (split > 1 ? 1.0 + 0.12 * split + 8e-7 * split * t * n : 0.0);
            if (best.bn == 0 || us < best_us) {
                best_us = us;
                best = BlockPlan{bn, static_cast<int>(split), static_cast<int>(split_kb), 0};
            }
        }
    }
    if (best.split > 1) best.part_bytes = static_cast<size_t>(best.split) * t * cdiv(n, 8) * 8 * 4;
    return best;
}

int launch_block(const CallContext& c, const BlockProduct& b, const BlockPlan& plan, float* part, cudaStream_t st,
                 int* launches) {
    Params p{};
    p.t = static_cast<int32_t>(b.t);
    p.n = static_cast<int32_t>(b.n);
    p.kbs = static_cast<int32_t>(cdiv(b.k, kBlock));
    p.tiles_t = static_cast<int32_t>(cdiv(b.t, kRows));
    p.tiles_n = static_cast<int32_t>(cdiv(b.n, plan.bn));
    p.split = plan.split;
    p.inv_split = 1.0f / static_cast<float>(p.split);
    p.inv_t = 1.0f / static_cast<float>(p.tiles_t);
    p.split_kb = plan.split_kb;
    p.x_scales = b.x_scales;
    p.xs_row = b.xs_row;
    p.xs_block = b.xs_block;
    p.w_scales = b.w_scales;
    p.ldws = b.ldws;
    p.bias = b.bias;
    p.act = b.act;
    p.residual = b.residual;
    p.ldr = b.ldr;
    p.y = b.y;
    p.ldy = b.ldy;
    auto aligned = [&](const void* q, int64_t ld) {
        return b.dtype == SGEMM_F32 ? rows_aligned<float>(q, ld) : rows_aligned<bf16>(q, ld);
    };
    p.vec = aligned(b.y, b.ldy) && aligned(b.residual, b.ldr) && aligned(b.bias, 0);
    p.part = plan.split > 1 ? part : nullptr;
    p.ldp = cdiv(b.n, 8) * 8;
    p.timeout_ns = c.timeout_ns;
    p.status = c.status;
    p.debug_flags = c.debug_flags;
    CUtensorMap m[2] = {};
    if (b.k > 0) {
        int rc;
        if ((rc = call_encode_u8(&m[0], b.x, b.k, b.t, b.ldx, kRows))) return rc;
        if ((rc = call_encode_u8(&m[1], b.w, b.k, b.n, b.ldw, static_cast<uint32_t>(plan.bn)))) return rc;
    }
    auto go = [&](auto zero) {
        using T = decltype(zero);
        cudaError_t e;
        switch (plan.bn) {
            case 64: e = run<64, T>(m, p, c.sms, st); break;
            case 128: e = run<128, T>(m, p, c.sms, st); break;
            default: e = run<256, T>(m, p, c.sms, st); break;
        }
        if (e != cudaSuccess || p.part == nullptr) return e;
        return launch_kernel(true, block_sum_kernel<T>, dim3(static_cast<unsigned>(cdiv(b.t * (p.ldp / 8), 256))), dim3(256),
                             0, st, p);
    };
    const cudaError_t e = b.dtype == SGEMM_F32 ? go(float()) : go(bf16());
    if (e != cudaSuccess) return call_fail_cuda(e, "block product");
    *launches += plan.split > 1 ? 2 : 1;
    return 0;
}

}  // namespace pg
