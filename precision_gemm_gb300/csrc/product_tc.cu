// The layer products (layers.h, struct Product) on the tensor cores: tcgen05 on SM
// pairs (cta_group::2, kind::f16), bfloat16 operands, FP32 accumulators in TMEM.
//
//     out[j][i] = epilogue(sum over k of A(i, k) B(j, k))
//
// A cluster of two CTAs computes a tile of 256 i x BN j: the feature direction i,
// which is contiguous in out, lies along TMEM lanes, so a warp's 32 lanes store 32
// neighbouring results and a narrow BN serves few rows (a decoding step, an
// expert's short list) without wasted weight traffic.  CTA r of the pair stages i
// rows [128 r, 128 r + 128) of A and j rows [r BN/2, ...) of B per 64-deep k block;
// one thread of CTA 0 issues the MMAs of both.
//
// Operands lie in shared memory in 128-byte swizzled rows of 64 values, either way
// round: K-major (rows along k) or MN-major (rows along i or j, one per k), so that
// y = x w^T, dx = dz w and dw = dz^T x all read their matrices as they are stored.
// In narrow tiles (BN <= 64) the rows of B can be gathered through a list by the TMA
// unit (tile::gather4), so that an expert's few tokens need no copy.  Wide tiles read
// rows that were copied together first: a gather of four 128-byte pieces takes the unit
// 88 cycles, hidden behind the weights' time in narrow tiles only (65536 x 1024 x 2048,
// 64 experts: 0.70 ms gathered by the TMA unit, 0.43 ms by 16-byte asynchronous copies
// of four more warps, 0.18 ms plus a copy of 0.05 ms).
//
// float32 operands come as three bfloat16 parts x = x0 + x1 + x2 (pack_kernel), whose
// six products of weight 2^-16 and above, the smallest first, are summed over a chunk
// of k in one accumulator.  The tensor core truncates its FP32 sums (an error of up to
// 2^-23 of the running sum per addition of 16 k, all one way), so a chunk is kept to 512 k
// and the chunks are added in registers, rounded to nearest, by the epilogue warps.
// bfloat16 sums are kept to chunks of 16384 k, which lose at most 2^-13 of the terms'
// magnitudes, a sixteenth of what rounding the result may.
//
// Warp roles as in tc2_kernel.cu: warp 0 loads, warp 1 issues MMAs, warps 2-9 drain
// TMEM (double-buffered: a unit's epilogue overlaps the next unit's MMAs).  The kernel
// is persistent; a unit is (tile, K slice).  With few tiles each tile's k is cut into
// slices; every slice stores its block, and sum_slices_kernel adds the blocks in slice
// order on all SMs (100 x 100 x 30000 bfloat16: 11 us, 27 when the slice that arrived last
// added them; 16 rows of 2048 x 8192: 9.5 and 14.4).
#include <algorithm>
#include <cstring>
#include <type_traits>

#include "layers.h"
#include "pair.cuh"
#include "ptx.cuh"

namespace pg {
namespace {

constexpr int kBK = 64;        // k per ring slot (128-byte rows)
constexpr int kChunkF32 = 512;     // k summed in one accumulator
constexpr int kChunkBf16 = 16384;
constexpr int kBI = 128;       // i per CTA
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kCols = 16;      // columns (j) that an epilogue warp takes at a time
constexpr int kGroupTiles = 8;  // rasterisation: tiles of j walked before the next tile of i

template <int BN>
struct Cfg {
    static constexpr int BNH = BN / 2;
    static constexpr int A_BYTES = kBI * kBK * 2;
    static constexpr int B_BYTES = BNH * kBK * 2;
    static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES_RAW = 200 * 1024 / STAGE_BYTES;
    static constexpr int STAGES = STAGES_RAW > 12 ? 12 : STAGES_RAW;
    static constexpr int TABLE_BYTES = 2 * (SGEMM_MAX_EXPERTS + 1) * 4 + 8;
    static constexpr int BAR_BYTES = (2 * STAGES + 5) * 8 + 16;
    static constexpr size_t SMEM = 1024 + static_cast<size_t>(STAGES) * STAGE_BYTES + TABLE_BYTES + BAR_BYTES;
    static constexpr uint32_t TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr int CHUNKS = BN / kCols;  // column chunks of a tile
    static constexpr int MINE = CHUNKS / 2;    // of one epilogue warp
    static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "slots need 1 KiB alignment");
    static_assert(TABLE_BYTES % 8 == 0, "barriers need 8-byte alignment");
};

struct Params {
    int32_t ni, nj, nk;
    int32_t groups;
    const int32_t* offsets;
    int32_t rows_on_k;
    int32_t a_mn, b_mn;
    int32_t segs;          // products of parts: 1 (bfloat16) or 6 (float32)
    int32_t chunk_kb;      // k blocks per accumulation chunk
    int32_t split, split_kb;  // K slices of the tiles from split_from on (1: none) ...
    int32_t halved;           // ... or their two halves along j, each a unit of its own
    int32_t split_from;
    int32_t a_z, b_z;      // third coordinates per part
    const int32_t* list;   // rows of B gathered: row r is list[r] / top (null: not gathered)
    int32_t top;
    int32_t a_rows, b_rows;  // rows per part
    int32_t a_oob, b_oob;    // a row past the matrix: reads as zeros
    int32_t tiles_i, tiles_j;  // tiles_j: of one group (rows_on_k) or unused
    const void* bias;
    int32_t act;
    const void* residual;
    int64_t ldr;
    void* out;
    int64_t ldo, out_stride;
    void* preact;
    int64_t ldz;
    int32_t out_f32;
    float* part;  // the slices' blocks
    int4* info;   // {tiles cut in slices}, then of each {i0, j0, j_end, group}
    uint64_t timeout_ns;
    int* status;
    int32_t debug_flags;
};

// The parts of A and B in segment s of a float32 product, the smallest terms first.
__device__ __forceinline__ int a_part(int s, int segs) { return segs == 1 ? 0 : (0x201100 >> (4 * (5 - s))) & 15; }
__device__ __forceinline__ int b_part(int s, int segs) { return segs == 1 ? 0 : (0x021010 >> (4 * (5 - s))) & 15; }

// Columns jb .. jb + N of a tile, sums v, for this thread's i < ni; `jn` of them are rows
// of out.
template <typename T, typename TO, int N>
__device__ __forceinline__ void finish(const Params& p, float (&v)[N], float bias, int64_t out_base, int64_t i,
                                       int64_t jb, int jn) {
    float r[N];
    if (p.residual) {
        const T* src = static_cast<const T*>(p.residual) + jb * p.ldr + i;
        const int64_t ld = p.ldr;
#pragma unroll
        for (int t = 0; t < N; ++t, src += ld) r[t] = t < jn ? to_float(*src) : 0.0f;
    }
#pragma unroll
    for (int t = 0; t < N; ++t) v[t] += bias;
    if (p.preact) {
        T* dst = static_cast<T*>(p.preact) + jb * p.ldz + i;
        const int64_t ld = p.ldz;
#pragma unroll
        for (int t = 0; t < N; ++t, dst += ld)
            if (t < jn) *dst = from_float<T>(v[t]);
    }
    with_act(p.act, [&](auto act) {
#pragma unroll
        for (int t = 0; t < N; ++t) v[t] = act_value<decltype(act)::value, std::is_same<T, bf16>::value>(v[t]);
    });
    if (p.residual) {
#pragma unroll
        for (int t = 0; t < N; ++t) v[t] += r[t];
    }
    TO* dst = static_cast<TO*>(p.out) + out_base + jb * p.ldo + i;
    const int64_t ld = p.ldo;
    if (jn >= N) {
#pragma unroll
        for (int t = 0; t < N; ++t, dst += ld) *dst = from_float<TO>(v[t]);
    } else {
#pragma unroll
        for (int t = 0; t < N; ++t, dst += ld)
            if (t < jn) *dst = from_float<TO>(v[t]);
    }
}

// F32: float32 operands in three parts, accumulated in chunks.
template <int BN, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    product_tc_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmAg, const __grid_constant__ CUtensorMap tmBg,
                      const __grid_constant__ CUtensorMap tmA16, const __grid_constant__ CUtensorMap tmB16,
                      const Params p) {
    using C = Cfg<BN>;
    using T = typename std::conditional<F32, float, bf16>::type;
    constexpr int S = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem_1024(smem_raw);
    int32_t* off = reinterpret_cast<int32_t*>(smem + S * C::STAGE_BYTES);  // first row of each group
    int32_t* pre = off + SGEMM_MAX_EXPERTS + 1;                            // first tile of each group
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S * C::STAGE_BYTES + C::TABLE_BYTES);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + 2 * S + 5);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    const uint32_t full0 = smem_u32(bars);
    const uint32_t empty0 = smem_u32(bars + S);
    const uint32_t acc_full0 = smem_u32(bars + 2 * S);
    const uint32_t acc_empty0 = smem_u32(bars + 2 * S + 2);
    const uint32_t mma_done = smem_u32(bars + 2 * S + 4);

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // known to be uniform
    const int lane = threadIdx.x & 31;
    const uint32_t rank = __shfl_sync(0xffffffffu, cluster_rank(), 0);
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1;
    const int pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full0 + 8 * s, 1);
            mbar_init(empty0 + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full0 + 8 * b, 1);
            mbar_init(acc_empty0 + 8 * b, 2 * kEpiWarps);
        }
        mbar_init(mma_done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(C::TMEM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    // The groups' rows and tiles.  Whatever the offsets hold, 0 <= off[g] <= off[g + 1] <= rows.
    const int rows = p.rows_on_k ? p.nk : p.nj;
    if (warp == 2) {
        int tiles = 0, last = 0;
        for (int g0 = 0; g0 < p.groups; g0 += 32) {
            const int g = g0 + lane;
            int first = 0, end = rows;
            if (p.offsets && g < p.groups) {
                first = min(max(p.offsets[g], 0), rows);
                end = min(max(p.offsets[g + 1], 0), rows);
            }
            // running maximum: no group starts before the one before it ends
            int top = max(first, last);
            for (int o = 1; o < 32; o <<= 1) top = max(top, __shfl_up_sync(0xffffffffu, top, o));
            first = top;
            const int next = __shfl_down_sync(0xffffffffu, first, 1);
            if (p.offsets && lane < 31 && g + 1 < p.groups) end = next;
            end = max(end, first);
            const int mine = g < p.groups ? (end - first + BN - 1) / BN : 0;
            int sum = mine;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            if (g < p.groups) {
                off[g] = first;
                pre[g] = tiles + sum - mine;
                if (g == p.groups - 1) off[p.groups] = end;
            }
            tiles += __shfl_sync(0xffffffffu, sum, 31);
            last = __shfl_sync(0xffffffffu, end, 31);
        }
        if (lane == 0) pre[p.groups] = tiles;
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // every CTA's barriers and TMEM exist before any cross-CTA traffic
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_holder, 0);
    const int tiles_j = p.rows_on_k ? p.tiles_j * p.groups : pre[p.groups];
    const int tiles = tiles_j * p.tiles_i;
    const int cuts = p.halved ? 2 : p.split;
    const int whole = cuts > 1 ? min(p.split_from, tiles) : tiles;  // tiles of one unit, first
    const int units = whole + (tiles - whole) * cuts;

    struct Unit {
        int tile, slice, g;  // tile counted from `whole` on, -1 for a unit of one slice
        int i0, j0, j_end;   // j_end: of the group (of the half)
        int n;               // width of its MMAs
        int k0, k_end;       // rows_on_k: the group's rows; else 0 and nk
        int kb0, nkb;        // this slice's k blocks
    };
    auto unit_of = [&](int u) {
        Unit x;
        // the slices of a tile are neighbours, so that they run at one time
        const int cut = u < whole ? 0 : (u - whole) % cuts;
        const int tile = u < whole ? u : whole + (u - whole) / cuts;
        x.tile = u < whole || p.halved ? -1 : tile - whole;
        x.slice = p.halved ? 0 : cut;
        int tj, ti;
        if (p.rows_on_k) {
            const int per = p.tiles_j * p.tiles_i;
            x.g = tile / per;
            tile_coords(tile - x.g * per, p.tiles_j, p.tiles_i, kGroupTiles, tj, ti);
            x.j0 = tj * BN;
            x.j_end = p.nj;
            x.k0 = off[x.g];
            x.k_end = off[x.g + 1];
        } else {
            tile_coords(tile, tiles_j, p.tiles_i, kGroupTiles, tj, ti);
            int lo = 0, hi = p.groups - 1;  // the last group whose first tile is at or before tj
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pre[mid] <= tj)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            x.g = lo;
            x.j0 = off[lo] + (tj - pre[lo]) * BN;
            x.j_end = off[lo + 1];
            x.k0 = 0;
            x.k_end = p.nk;
        }
        x.i0 = ti * (2 * kBI);
        if (p.halved && u >= whole) {
            x.j0 += cut * (BN / 2);
            x.j_end = min(x.j_end, x.j0 + BN / 2);
        }
        // the narrowest MMAs that hold the unit's columns (B read in groups of 64 columns: 128 at least)
        x.n = BN;
        while (x.n > (p.b_mn ? 128 : 32) && x.j_end - x.j0 <= x.n / 2) x.n /= 2;
        const int kb_total = (x.k_end - x.k0 + kBK - 1) / kBK;
        x.kb0 = x.tile < 0 ? 0 : x.slice * p.split_kb;
        x.nkb = x.tile < 0 ? kb_total : max(min(x.kb0 + p.split_kb, kb_total) - x.kb0, 0);
        if (x.j0 >= x.j_end) x.nkb = 0;  // a half past the end
        return x;
    };

    // The accumulator that a chunk takes (`next`) and the phase bits of both, kept alike by the MMA
    // issuer and the epilogue.  float32's many chunks alternate.  bfloat16's first chunk keeps its
    // accumulator until the unit ends, the others all take the second and are added to it there.
    auto take_buffer = [](int& next, uint32_t& phases, bool first) {
        phases ^= 1u << next;
        if (F32 || first) next ^= 1;
    };

    if (warp == 0) {
        // ---------------- TMA loader (both CTAs) ----------------
        if (!(p.debug_flags & 1)) {
            const uint32_t full_leader0 = map_to_rank(full0, 0);
            int it = 0, slot_i = 0;
            uint32_t phase = 1;
            bool ok = true;
            // The warp runs as one, an elected lane issues.  LISTED: some rows are named one by one
            // (gathered rows of B, or lists that may end inside a k block), four by each lane.
            auto load = [&](auto listed) {
                constexpr bool LISTED = decltype(listed)::value;
                for (int u = pair; u < units && ok; u += pairs) {
                    Unit x = unit_of(u);
                    // known to be uniform from here on: operands of the copies
                    x.i0 = __shfl_sync(0xffffffffu, x.i0, 0);
                    x.j0 = __shfl_sync(0xffffffffu, x.j0, 0);
                    x.g = __shfl_sync(0xffffffffu, x.g, 0);
                    x.k0 = __shfl_sync(0xffffffffu, x.k0, 0);
                    x.k_end = __shfl_sync(0xffffffffu, x.k_end, 0);
                    x.kb0 = __shfl_sync(0xffffffffu, x.kb0, 0);
                    x.nkb = __shfl_sync(0xffffffffu, x.nkb, 0);
                    x.n = __shfl_sync(0xffffffffu, x.n, 0);
                    const int ia = x.i0 + kBI * static_cast<int>(rank);
                    const int jb = x.j0 + x.n / 2 * static_cast<int>(rank);
                    const bool gather = LISTED && p.list != nullptr;
                    int4 rows_b = make_int4(0, 0, 0, 0);  // this lane's four gathered rows of B
                    if (gather && lane < C::BNH / 4) {
                        int* y = &rows_b.x;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int r = jb + 4 * lane + q;
                            const int64_t v = r < x.j_end ? gathered_row(p.list, p.top, r, p.b_rows) : -1;
                            y[q] = v >= 0 ? static_cast<int>(v) : p.b_oob;
                        }
                    }
                    for (int c0 = 0; c0 < x.nkb && ok; c0 += p.chunk_kb) {
                        const int c1 = min(c0 + p.chunk_kb, x.nkb);
                        for (int s = 0; s < p.segs && ok; ++s) {
                            const int pa = a_part(s, p.segs), pb = b_part(s, p.segs);
                            const int z_a = p.rows_on_k ? pa * p.a_z : pa * p.a_z + x.g;
                            const int z_b = pb * p.b_z;
                            for (int kb = c0; kb < c1; ++kb, ++it) {
                                ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty0 + 8 * slot_i, phase, p.timeout_ns,
                                                                               abort_flag));
                                if (!ok) {
                                    if (lane == 0) raise_abort(abort_flag, p.status);
                                    break;
                                }
                                const int kc = x.k0 + (x.kb0 + kb) * kBK;
                                // A group's rows may end inside this block.  The rows past them must read as
                                // zeros, not as the next group's: whole runs of 16 come in boxes of 16 rows,
                                // the last, partial one row by row, and the MMAs stop after it.
                                const int left = LISTED && p.rows_on_k ? x.k_end - kc : kBK;
                                const bool ragged = LISTED && left < kBK;
                                if (leader && lane == 0)
                                    mbar_arrive_expect_tx(full0 + 8 * slot_i,
                                                          2 * (ragged ? C::STAGE_BYTES / 4 * ((left + 15) / 16)
                                                                      : C::STAGE_BYTES));
                                const uint32_t bar = full_leader0 + 8 * slot_i;
                                const uint32_t slot = smem_u32(smem) + slot_i * C::STAGE_BYTES;
                                const uint32_t slot_b = slot + C::A_BYTES;
                                if (ragged) {
                                    const int runs = left / 16;
                                    if (lane < 16) {
                                        // run q of 64 columns: A's two groups, then B's
                                        const int q = lane >> 2, h = lane & 1;
                                        if (q < runs && (lane & 2) == 0)
                                            tma_load_3d_pair(slot + 8192 * h + 2048 * q, &tmA16, ia + 64 * h,
                                                             kc + 16 * q, z_a, bar);
                                        else if (q < runs && h < C::BNH / 64)
                                            tma_load_3d_pair(slot_b + 8192 * h + 2048 * q, &tmB16, jb + 64 * h,
                                                             kc + 16 * q, z_b, bar);
                                    } else if (left % 16 != 0) {
                                        const int q = (lane >> 2) & 3, h = lane & 1, r = kc + 16 * runs + 4 * q;
                                        const bool of_a = (lane & 2) == 0;
                                        int4 y;
                                        int* py = &y.x;
#pragma unroll
                                        for (int k = 0; k < 4; ++k)
                                            py[k] = r + k < x.k_end ? r + k + (of_a ? pa * p.a_rows : pb * p.b_rows)
                                                                    : (of_a ? p.a_oob : p.b_oob);
                                        const uint32_t at = 8192 * h + 2048 * runs + 512 * q;
                                        if (of_a)
                                            tma_gather4_pair(slot + at, &tmAg, ia + 64 * h, y, bar);
                                        else if (h < C::BNH / 64)
                                            tma_gather4_pair(slot_b + at, &tmBg, jb + 64 * h, y, bar);
                                    }
                                    __syncwarp();
                                } else {
                                    if (p.a_mn) {
                                        tma_load_3d_pair_warp(slot, &tmA, ia, kc, z_a, bar);
                                        tma_load_3d_pair_warp(slot + 8192, &tmA, ia + 64, kc, z_a, bar);
                                    } else {
                                        tma_load_3d_pair_warp(slot, &tmA, kc, ia, z_a, bar);
                                    }
                                    if (p.b_mn) {
#pragma unroll
                                        for (int h = 0; h < C::BNH / 64; ++h)
                                            tma_load_3d_pair_warp(slot_b + 8192 * h, &tmB, jb + 64 * h, kc, z_b, bar);
                                    } else if (!gather) {
                                        tma_load_3d_pair_warp(slot_b, &tmB, kc, jb, z_b, bar);
                                    }
                                }
                                if (gather && lane < C::BNH / 4)
                                    tma_gather4_pair(slot_b + 512 * lane, &tmBg, kc, rows_b, bar);
                                if (++slot_i == S) {
                                    slot_i = 0;
                                    phase ^= 1;
                                }
                            }
                        }
                    }
                }
            };
            if (p.list != nullptr || (p.rows_on_k && p.offsets != nullptr)) {
                load(std::true_type());
            } else {
                load(std::false_type());
            }
            if (lane == 0) pdl_trigger();
            if (leader && lane == 0) {
                // Let every copy of the pair land before the CTAs may retire (CTA 0's
                // full barriers count both CTAs' bytes).
                for (int j = max(0, it - S); j < it; ++j)
                    mbar_wait_bounded(full0 + 8 * (j % S), (j / S) & 1, p.timeout_ns, nullptr);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer (CTA 0 of the pair) ----------------
        // The warp runs as one: what the MMAs are given is uniform, and one lane issues.
        if (leader) {
            // K-major: 8-row atoms 1 KiB apart, a k-step of 16 is 32 bytes further along the rows.
            // MN-major: 64-column groups 8 KiB apart, 8-k atoms 1 KiB apart, a k-step 2 KiB further.
            const uint32_t slot0 = smem_u32(smem);
            const uint64_t a_desc0 = smem_desc(slot0, p.a_mn ? 8192 : 16, 1024, kSwizzle128B);
            const uint64_t b_desc0 = smem_desc(slot0 + C::A_BYTES, p.b_mn ? 8192 : 16, 1024, kSwizzle128B);
            const uint32_t a_step = p.a_mn ? 128 : 2, b_step = p.b_mn ? 128 : 2;
            const bool ragged = p.rows_on_k && p.offsets != nullptr;
            int slot_i = 0, next = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true;
            for (int u = pair; u < units && ok; u += pairs) {
                const Unit x = unit_of(u);
                const int nkb = __shfl_sync(0xffffffffu, x.nkb, 0);
                const int rows_left = __shfl_sync(0xffffffffu, x.k_end - x.k0 - x.kb0 * kBK, 0);  // from kb0 on
                const uint32_t idesc =
                    idesc_bf16(2 * kBI, __shfl_sync(0xffffffffu, x.n, 0), p.a_mn != 0, p.b_mn != 0);
                for (int c0 = 0; c0 < nkb && ok; c0 += p.chunk_kb) {
                    const int steps = (min(c0 + p.chunk_kb, nkb) - c0) * p.segs;
                    const int buf = next;
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(acc_empty0 + 8 * buf, ((acc_phase >> buf) & 1) ^ 1,
                                                                   p.timeout_ns, abort_flag));
                    if (!ok) break;
                    take_buffer(next, acc_phase, c0 == 0);
                    tc_fence_after_sync();
                    const uint32_t d = tmem + buf * BN;
                    uint32_t accumulate = 0;
                    for (int kb = 0; kb < steps; ++kb) {
                        ok = __all_sync(0xffffffffu,
                                        mbar_wait_bounded(full0 + 8 * slot_i, phase, p.timeout_ns, abort_flag));
                        if (!ok) break;
                        tc_fence_after_sync();
                        const uint32_t o = static_cast<uint32_t>(slot_i * C::STAGE_BYTES) >> 4;
                        // a group's last block stops at its last run of 16 rows
                        const int left = ragged ? rows_left - (kb % (min(c0 + p.chunk_kb, nkb) - c0) + c0) * kBK : kBK;
#pragma unroll
                        for (int kk = 0; kk < kBK / 16; ++kk) {
                            if (16 * kk >= left) break;
                            mma_bf16_pair_warp(d, a_desc0 + (o + kk * a_step), b_desc0 + (o + kk * b_step), idesc,
                                               accumulate);
                            accumulate = 1;
                        }
                        mma_commit_pair_warp(empty0 + 8 * slot_i);
                        if (++slot_i == S) {
                            slot_i = 0;
                            phase ^= 1;
                        }
                    }
                    if (ok) mma_commit_pair_warp(acc_full0 + 8 * buf);
                }
            }
            if (!ok && lane == 0) raise_abort(abort_flag, p.status);
            mma_commit_pair_local_warp(mma_done);  // every MMA issued here has completed
            mbar_wait_bounded(mma_done, 0, p.timeout_ns, nullptr);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue (warps 2..9, both CTAs) ----------------
        const int q = warp & 3;             // TMEM lane quarter this warp may access
        const int half = (warp - 2) >> 2;   // it takes every other 16 columns
        const uint32_t acc_empty_leader0 = map_to_rank(acc_empty0, 0);
        const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
        const int epi = warp - 2;
        // rows of no group are zero
        if (!p.rows_on_k && p.offsets) {
            const int used = off[p.groups];
            for (int64_t j = used + blockIdx.x * kEpiWarps + epi; j < p.nj; j += gridDim.x * kEpiWarps) {
                for (int i = lane; i < p.ni; i += 32) {
                    if (!F32 && !p.out_f32)
                        static_cast<T*>(p.out)[j * p.ldo + i] = from_float<T>(0.0f);
                    else
                        static_cast<float*>(p.out)[j * p.ldo + i] = 0.0f;
                    if (p.preact) static_cast<T*>(p.preact)[j * p.ldz + i] = from_float<T>(0.0f);
                }
            }
        }
        if (p.part && blockIdx.x == 0 && epi == 0 && lane == 0) p.info[0] = make_int4(tiles - whole, 0, 0, 0);
        float bias = 0.0f;  // of the unit's group and this thread's i
        auto finish_chunk = [&](const Unit& x, float(&v)[kCols], int c) {
            const int64_t i = x.i0 + kBI * rank + 32 * q + lane;
            if (i >= p.ni) return;
            const int64_t jb = x.j0 + kCols * c;
            const int jn = x.j_end - x.j0 - kCols * c;
            const int64_t base = p.rows_on_k ? x.g * p.out_stride : 0;
            if (F32 || !p.out_f32)
                finish<T, T>(p, v, bias, base, i, jb, jn);
            else
                finish<T, float>(p, v, bias, base, i, jb, jn);
        };
        int next = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int u = pair; u < units && ok; u += pairs) {
            const Unit x = unit_of(u);
            const int cols = min(BN, x.j_end - x.j0);
            // this slice's block: [column][256 i]
            float* block = x.tile >= 0 ? p.part + (static_cast<int64_t>(x.tile) * p.split + x.slice) * (2 * kBI * BN) +
                                             kBI * rank + 32 * q + lane
                                       : nullptr;
            const int64_t i = x.i0 + kBI * rank + 32 * q + lane;
            if (p.bias && i < p.ni) bias = to_float(static_cast<const T*>(p.bias)[static_cast<int64_t>(x.g) * p.ni + i]);
            if (p.residual && i - lane < p.ni) {
                // the residual comes into L2 while the MMAs run: lane t asks for column t's line
                for (int t = kCols * half + lane % kCols + 2 * kCols * (lane / kCols); t < cols; t += 4 * kCols)
                    prefetch_l2(static_cast<const T*>(p.residual) + (x.j0 + t) * p.ldr + i - lane);
            }
            const bool any = x.nkb > 0;  // a sum without k (k = 0, an expert without rows) is zero
            auto wait_sums = [&](bool first) {  // the next chunk's sums; their buffer
                const int buf = next;
                ok = __all_sync(0xffffffffu,
                                mbar_wait_bounded(acc_full0 + 8 * buf, (acc_phase >> buf) & 1, p.timeout_ns, abort_flag));
                if (!ok && lane == 0) raise_abort(abort_flag, p.status);
                tc_fence_after_sync();
                take_buffer(next, acc_phase, first);
                return buf;
            };
            auto free_sums = [&](int buf) {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_relaxed(acc_empty_leader0 + 8 * buf);
            };
            int buf = 0;
            if (F32 && x.nkb > p.chunk_kb) {
                // Add the chunks; the whole sum goes back to the last one's columns, where the loop
                // below finds it as it finds a single chunk's (kept in registers, the sums would
                // leave it too few to have its loads in flight together).
                float acc[C::MINE][kCols];
#pragma unroll
                for (int m = 0; m < C::MINE; ++m)
#pragma unroll
                    for (int t = 0; t < kCols; ++t) acc[m][t] = 0.0f;
                for (int c0 = 0; c0 < x.nkb; c0 += p.chunk_kb) {
                    buf = wait_sums(c0 == 0);
                    if (!ok) break;
#pragma unroll
                    for (int m = 0; m < C::MINE; ++m) {
                        if (kCols * (half + 2 * m) < cols) {
                            uint32_t v[kCols];
                            __syncwarp();
                            tmem_ld_32x32b_x16(lane_base + buf * BN + kCols * (half + 2 * m), v);
                            tmem_wait_ld();
#pragma unroll
                            for (int t = 0; t < kCols; ++t) acc[m][t] += __uint_as_float(v[t]);
                        }
                    }
                    if (c0 + p.chunk_kb < x.nkb) free_sums(buf);
                }
                if (!ok) break;
#pragma unroll
                for (int m = 0; m < C::MINE; ++m) {
                    if (kCols * (half + 2 * m) < cols) {
                        uint32_t v[kCols];
#pragma unroll
                        for (int t = 0; t < kCols; ++t) v[t] = __float_as_uint(acc[m][t]);
                        __syncwarp();
                        tmem_st_32x32b_x16(lane_base + buf * BN + kCols * (half + 2 * m), v);
                    }
                }
                tmem_wait_st();
            } else if (any) {
                buf = wait_sums(true);
                if (!ok) break;
                // bfloat16: the further chunks are added to the first one's columns, 16 at a time (with a
                // whole tile's sums in registers the kernel is slower where k is short too: dw of 32768
                // rows of 64 experts 149 us, then 173)
#pragma unroll 1
                for (int c0 = p.chunk_kb; !F32 && c0 < x.nkb; c0 += p.chunk_kb) {
                    const int more = wait_sums(false);
                    if (!ok) break;
#pragma unroll 1
                    for (int c = half; kCols * c < cols; c += 2) {
                        uint32_t v[kCols], sum[kCols];
                        __syncwarp();
                        tmem_ld_32x32b_x16(lane_base + more * BN + kCols * c, v);
                        tmem_ld_32x32b_x16(lane_base + buf * BN + kCols * c, sum);
                        tmem_wait_ld();
#pragma unroll
                        for (int t = 0; t < kCols; ++t)
                            sum[t] = __float_as_uint(__uint_as_float(sum[t]) + __uint_as_float(v[t]));
                        __syncwarp();
                        tmem_st_32x32b_x16(lane_base + buf * BN + kCols * c, sum);
                    }
                    tmem_wait_st();
                    free_sums(more);
                }
                if (!ok) break;
            }
#pragma unroll 1
            for (int c = half; kCols * c < cols; c += 2) {
                float f[kCols];
                __syncwarp();
                if (any) {
                    uint32_t v[kCols];
                    tmem_ld_32x32b_x16(lane_base + buf * BN + kCols * c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int t = 0; t < kCols; ++t) f[t] = __uint_as_float(v[t]);
                } else {
#pragma unroll
                    for (int t = 0; t < kCols; ++t) f[t] = 0.0f;
                }
                if (block) {
#pragma unroll
                    for (int t = 0; t < kCols; ++t) block[(kCols * c + t) * (2 * kBI)] = f[t];
                } else {
                    finish_chunk(x, f, c);
                }
            }
            if (any) free_sums(buf);
            if (block && x.slice == 0 && rank == 0 && epi == 0 && lane == 0)
                p.info[1 + x.tile] = make_int4(x.i0, x.j0, x.j_end, x.g);
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();  // no CTA leaves while its peer may still read its shared memory or barriers
    if (warp == 1) {
        tc_fence_after_sync();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS)
                     : "memory");
    }
}

// The tiles that were cut along k: thread i of a block adds the slices of kSumCols columns
// in their order and finishes them.  The tiles' places are checked against the matrix, since
// a product that gave up (a wait that expired) may not have written them.
constexpr int kSumCols = 4;
template <bool F32>
__global__ void __launch_bounds__(2 * kBI) sum_slices_kernel(const Params p, int bn, int most) {
    using T = typename std::conditional<F32, float, bf16>::type;
    pdl_trigger();
    pdl_wait();
    const int per = bn / kSumCols, tile = blockIdx.x / per, c0 = (blockIdx.x - tile * per) * kSumCols;
    if (tile >= min(p.info[0].x, most)) return;
    const int4 at = p.info[1 + tile];
    const int64_t i = static_cast<int64_t>(at.x) + threadIdx.x;
    const int jn = at.z - at.y - c0;
    if (at.x < 0 || i >= p.ni || at.y < 0 || at.z > p.nj || jn <= 0 || at.w < 0 || at.w >= p.groups) return;
    const float* src = p.part + static_cast<int64_t>(tile) * p.split * (2 * kBI * bn) + c0 * (2 * kBI) + threadIdx.x;
    float v[kSumCols] = {};
    for (int s0 = 0; s0 < p.split; s0 += 8) {
        float b[8][kSumCols];
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int t = 0; t < kSumCols; ++t)
                b[s][t] = s0 + s < p.split
                              ? __ldcg(src + static_cast<int64_t>(s0 + s) * (2 * kBI * bn) + t * (2 * kBI))
                              : 0.0f;
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int t = 0; t < kSumCols; ++t) v[t] += b[s][t];
    }
    const float bias =
        p.bias ? to_float(static_cast<const T*>(p.bias)[static_cast<int64_t>(at.w) * p.ni + i]) : 0.0f;
    const int64_t base = p.rows_on_k ? at.w * p.out_stride : 0;
    if (F32 || !p.out_f32)
        finish<T, T>(p, v, bias, base, i, at.y + c0, jn);
    else
        finish<T, float>(p, v, bias, base, i, at.y + c0, jn);
}

// x = x0 + x1 + x2 with x0 = bf16(x), x1 = bf16(x - x0), x2 = bf16(x - x0 - x1); both
// differences are exact in FP32, so the three parts hold x's 24 bits (down to
// bfloat16's smallest subnormal, 2^-133).  Of an infinity x0 is +-1 and x2 the
// infinity, which meets only the other operand's x0: its products are then those of
// FP32 (see split_tf32); NaN stays in x2.  bfloat16 rows are copied (PARTS 1).
// A thread takes eight columns of R rows: 16-byte accesses where the source allows
// them, R rows' loads in flight.  HBM-bound: 10 bytes moved per float32 element (64
// matrices of 1024 x 2048: 215 us, 6.2 TB/s).  blockIdx.y: the matrix.
struct PackJobs {
    PackJob job[2];
};
template <typename T, int PARTS, int R>
__global__ void __launch_bounds__(256) pack_kernel(const PackJobs jobs) {
    pdl_trigger();
    pdl_wait();
    const PackJob& j = jobs.job[blockIdx.y];
    const T* src = static_cast<const T*>(j.src);
    const int64_t rows = j.groups * j.per_group;
    const uint32_t eights = static_cast<uint32_t>((j.cols + 7) / 8);
    const int64_t items = (rows + R - 1) / R * eights;
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; q < items;
         q += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t r0 = items >> 32 ? q / eights : static_cast<uint32_t>(q) / eights;
        const int64_t c = (q - r0 * eights) * 8;
        const int valid = static_cast<int>(j.cols - c < 8 ? j.cols - c : 8);
        float v[R][8] = {};
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t r = r0 * R + k;
            if (r >= rows) break;
            if (j.list) {
                const int64_t s = gathered_row(j.list, j.top, r, j.src_rows);
                if (s >= 0) load8(src + s * j.ld + c, j.vec, valid, v[k]);
            } else {
                const int64_t g = j.groups == 1 ? 0 : r / j.per_group;
                load8(src + g * j.stride + (r - g * j.per_group) * j.ld + c, j.vec, valid, v[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t r = r0 * R + k;
            if (r < rows) store_parts8<PARTS>(j.dst + r * j.ldd + c, rows * j.ldd, v[k]);
        }
    }
}

// Listed bfloat16 rows copied together: a warp per row and 2048 columns, its 16-byte
// loads in flight together.  A row's last 16 bytes may reach past its columns, inside
// the 16-byte block of its last element; no product reads those.  Bound by the writes
// (65536 rows of 2048: 50 us, 5.4 TB/s).
__global__ void __launch_bounds__(256) copy_rows_kernel(const bf16* src, int64_t ld, int64_t rows, const int32_t* list,
                                                        int top, int64_t src_rows, bf16* dst, int64_t ldd, int eights) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x % 32;
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
    if (r >= rows) return;
    const int64_t s = gathered_row(list, top, r, src_rows);
    const int first = blockIdx.y * 256;
    const uint4* in = reinterpret_cast<const uint4*>(src + (s >= 0 ? s : 0) * ld) + first;
    uint4* out = reinterpret_cast<uint4*>(dst + r * ldd) + first;
    uint4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (s >= 0 && first + 32 * k + lane < eights) v[k] = in[32 * k + lane];
        else v[k] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (first + 32 * k + lane < eights) out[32 * k + lane] = v[k];
}

template <int BN, bool F32>
cudaError_t launch(const CUtensorMap (&m)[6], const Params& p, int64_t units, int num_sms, cudaStream_t st) {
    using C = Cfg<BN>;
    auto kern = product_tc_kernel<BN, F32>;
    static std::atomic<uint64_t> smem_set{0};
    cudaError_t e = set_smem_limit_once(smem_set, reinterpret_cast<const void*>(kern), static_cast<int>(C::SMEM));
    if (e != cudaSuccess) return e;
    // Clusters that are resident together (they must fit inside GPCs), asked once per device; a
    // persistent grid beyond them would run a second time around.
    static std::atomic<int> resident[64];
    int dev = 0;
    cudaGetDevice(&dev);
    int most = dev >= 0 && dev < 64 ? resident[dev].load() : 0;
    if (most <= 0) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3(2, 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = C::SMEM;
        if (cudaOccupancyMaxActiveClusters(&most, kern, &cfg) != cudaSuccess || most <= 0) {
            cudaGetLastError();
            most = num_sms / 2;
        }
        if (dev >= 0 && dev < 64) resident[dev] = most;
    }
    const int64_t clusters = std::max<int64_t>(1, std::min<int64_t>(units, most));
    return launch_kernel(true, kern, dim3(static_cast<unsigned>(2 * clusters)), dim3(kThreads), C::SMEM,
                         st, m[0], m[1], m[2], m[3], m[4], m[5], p);
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t region(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_pack(int dtype, const PackJob* jobs, int count, int num_sms, cudaStream_t st) {
    PackJobs all{};
    int64_t most = 0;
    for (int q = 0; q < count; ++q) {
        PackJob& j = all.job[q];
        j = jobs[q];
        j.vec = dtype == SGEMM_F32 ? rows_aligned<float>(j.src, j.ld) && (j.groups == 1 || j.stride % 4 == 0)
                                   : rows_aligned<bf16>(j.src, j.ld) && (j.groups == 1 || j.stride % 8 == 0);
        most = std::max(most, j.groups * j.per_group * cdiv(j.cols, 8));
    }
    const PackJob& j = all.job[0];
    // whole eights of a row exist where the rows are aligned and their stride covers them
    if (dtype == SGEMM_BF16 && count == 1 && j.list && j.vec && j.ld >= cdiv(j.cols, 8) * 8 && cdiv(j.cols, 8) <= 256 * 65535)
        return launch_kernel(true, copy_rows_kernel,
                             dim3(static_cast<unsigned>(cdiv(j.per_group, 8)), static_cast<unsigned>(cdiv(j.cols, 8 * 256))),
                             dim3(256), 0, st, static_cast<const bf16*>(j.src), j.ld, j.per_group, j.list, j.top,
                             j.src_rows, j.dst, j.ldd, static_cast<int>(cdiv(j.cols, 8)));
    // four rows per thread once that leaves each SM 2048 threads
    const int r = most / 4 >= int64_t(2048) * num_sms ? 4 : 1;
    const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(cdiv(cdiv(most, r), 256), 16 * num_sms))),
                    static_cast<unsigned>(count));
    auto kern = dtype == SGEMM_F32 ? (r == 4 ? pack_kernel<float, 3, 4> : pack_kernel<float, 3, 1>)
                                   : (r == 4 ? pack_kernel<bf16, 1, 4> : pack_kernel<bf16, 1, 1>);
    return launch_kernel(true, kern, grid, dim3(256), 0, st, all);
}

// Tile width, K slices and the last wave, by an estimate of the kernel's time in us:
//     waves * steps * step(bn) + end(bn) [+ kSplit + kBlockMB * MB of the slices' blocks]
// with one step per k block and product of parts.  Measured at 4864 x 4096 x 4096
// (whole waves at every width): a step of all pairs takes 0.34 us at 256 columns, 0.19
// at 128, 0.14 at 64 (operand feed: A's 128 rows per CTA are loaded whatever the width);
// the end is the last tile's epilogue, which no MMAs hide (most with a residual, whose
// reads it waits for); kSplit and kBlockMB are the adding kernel and the blocks' way to it.
// Against tiles that are not cut: 16 rows of 4096 x 4096 bfloat16 12.7 -> 8.8 us, of 2048 x
// 8192 21.6 -> 9.5; float32, 40 rows of 2048 x 2048 42 -> 20, 400 rows 43 -> 33, 700^3 18.3
// -> 16.9.  Tile widths: 1500 x 3000 x 777 float32 with residual takes 40 us from cold caches
// at 256 columns (72 tiles, one wave, whose epilogue nothing hides) as at 128 (two waves).
// Grouped rows are counted by their average length, since the lengths are known on the
// device alone.
TcPlan plan_tc(const Product& p, int num_sms, int force_bn, int force_split) {
    static constexpr double kSplit = 2.0, kBlockMB = 0.2;
    const int pairs = std::max(num_sms / 2, 1);
    const int64_t tiles_i = cdiv(p.ni, 2 * kBI), kb = cdiv(p.nk, kBK);
    const int64_t lists = p.rows_on_k ? 1 : std::max<int64_t>(1, std::min<int64_t>(p.groups, p.nj));
    const double segs = p.dtype == SGEMM_F32 ? 6.0 : 1.0;
    // groups that share out k hold a group's part of it each, on average
    const double steps = segs * (p.rows_on_k && p.groups > 1 ? std::max(1.0, static_cast<double>(kb) / p.groups) : kb);
    TcPlan best{};
    double best_us = 0.0;
    for (int bn : {256, 128, 64, 32}) {
        if (bn < 128 && !p.b.k_contiguous) break;
        if (force_bn && bn != (p.b.k_contiguous ? force_bn : std::max(force_bn, 128)) && force_bn <= 256) continue;
        const double step = bn == 256 ? 0.34 : (bn == 128 ? 0.19 : (bn == 64 ? 0.14 : 0.12));
        const double end = (bn == 256 ? 4.0 : (bn == 128 ? 2.0 : 1.0)) * (p.residual ? 3.0 : 1.0);
        const int64_t tiles = p.rows_on_k ? tiles_i * cdiv(p.nj, bn) * p.groups
                                          : tiles_i * lists * cdiv(cdiv(p.nj, lists), bn);
        TcPlan t{};
        t.bn = bn;
        t.split = 1;
        t.split_kb = static_cast<int>(std::max<int64_t>(kb, 1));
        // a last wave at most half full: its tiles' halves along j, whose MMAs of N = 128 take 0.56 of
        // the time (4096^3 bfloat16: cut in two along k 84.6 us, halves 76.7)
        const int64_t waves = cdiv(tiles, pairs), last = tiles % pairs;
        t.halved = bn == 256 && force_split == 0 && p.groups == 1 && waves > 1 && last > 0 && 2 * last <= pairs;
        t.whole = last;  // for now: the tiles of the last wave
        double us = (t.halved ? static_cast<double>(waves) - 0.44 : static_cast<double>(waves)) * steps * step + end;
        // K slices that fill one, two or three waves (not groups that share out k: their lengths differ)
        for (int64_t w = 1; w <= 3 && !(p.rows_on_k && p.groups > 1) && kb > 1; ++w) {
            const int64_t want = force_split > 0 ? std::min<int64_t>(force_split, kb)
                                                 : std::min<int64_t>(w * pairs / tiles, std::max<int64_t>(kb / 4, 1));
            if (want < 2) continue;
            const int64_t split_kb = cdiv(kb, want), split = cdiv(kb, split_kb);
            const double blocks_mb = static_cast<double>(tiles) * split * bn * (2 * kBI * 4) * 1e-6;
            const double cut_us =
                static_cast<double>(cdiv(tiles * split, pairs)) * segs * split_kb * step + end + kSplit + kBlockMB * blocks_mb;
            if (split > 1 && (force_split > 0 || cut_us < us)) {
                us = cut_us;
                t.split = static_cast<int>(split);
                t.split_kb = static_cast<int>(split_kb);
                t.halved = false;
            }
        }
        if (best.bn == 0 || us < best_us) {
            best = t;
            best_us = us;
        }
    }
    TcPlan t = best;
    const int64_t last = t.whole;
    t.tiles = p.rows_on_k ? tiles_i * cdiv(p.nj, t.bn) * p.groups
                          : tiles_i * (cdiv(p.nj, t.bn) + (p.groups > 1 ? lists : 0));
    t.whole = t.split > 1 ? 0 : (t.halved ? t.tiles - last : t.tiles);
    t.gather = t.bn <= 64 && !p.rows_on_k;
    if (t.split > 1) {
        t.part_bytes = region(static_cast<size_t>(t.tiles) * t.split * 2 * kBI * t.bn * 4);
        t.info_bytes = region(static_cast<size_t>(t.tiles + 1) * sizeof(int4));
    }
    return t;
}

// p.a and p.b: bfloat16 matrices that TMA can read (16-byte aligned, ld and stride
// multiples of 8), in `parts` parts one after another.
int launch_product_tc(const CallContext& c, const Product& p, const TcPlan& t, int parts, void* ws, cudaStream_t st,
                      int* launches) {
    Params q{};
    q.ni = static_cast<int32_t>(p.ni);
    q.nj = static_cast<int32_t>(p.nj);
    q.nk = static_cast<int32_t>(p.nk);
    q.groups = p.groups;
    q.offsets = p.offsets;
    q.rows_on_k = p.rows_on_k;
    q.a_mn = !p.a.k_contiguous;
    q.b_mn = !p.b.k_contiguous;
    q.segs = parts == 3 ? 6 : 1;
    q.chunk_kb = (parts == 3 ? kChunkF32 : kChunkBf16) / kBK;
    q.split = t.split;
    q.split_kb = t.split_kb;
    q.halved = t.halved;
    q.split_from = static_cast<int32_t>(t.whole);
    q.a_z = p.rows_on_k ? 1 : p.groups;
    q.b_z = 1;
    q.list = p.b.list;
    q.top = p.b.top;
    q.a_rows = static_cast<int32_t>(p.a.rows);
    q.b_rows = static_cast<int32_t>(p.b.rows);
    q.a_oob = static_cast<int32_t>(p.a.rows * parts);
    q.b_oob = static_cast<int32_t>(p.b.rows * parts);
    q.tiles_i = static_cast<int32_t>(cdiv(p.ni, 2 * kBI));
    q.tiles_j = static_cast<int32_t>(cdiv(p.nj, t.bn));
    q.bias = p.bias;
    q.act = p.act;
    q.residual = p.residual;
    q.ldr = p.ldr;
    q.out = p.out;
    q.ldo = p.ldo;
    q.out_stride = p.out_stride;
    q.preact = p.preact;
    q.ldz = p.ldz;
    q.out_f32 = p.out_f32;
    q.timeout_ns = c.timeout_ns;
    q.status = c.status;
    q.debug_flags = c.debug_flags;
    if (t.split > 1) {
        q.part = static_cast<float*>(ws);
        q.info = reinterpret_cast<int4*>(static_cast<char*>(ws) + t.part_bytes);
    }
    // Columns of each matrix.  Packed rows along i or j count as whole: boxes that reach past
    // a matrix load slower, and what lies there only meets results that are not stored.
    const int64_t cols_a = p.a.k_contiguous ? p.nk : (p.a.packed ? p.a.ld : p.ni);
    const int64_t cols_b = p.b.k_contiguous ? p.nk : (p.b.packed ? p.b.ld : p.nj);
    const int64_t z_a = (p.rows_on_k ? 1 : p.groups) * static_cast<int64_t>(parts);
    CUtensorMap m[6];
    int rc;
    if (p.nk == 0) {  // nothing is loaded: the maps stay unread
        std::memset(m, 0, sizeof m);
    } else {
        const uint32_t box_a = p.a.k_contiguous ? kBI : kBK, box_b = p.b.k_contiguous ? t.bn / 2 : kBK;
        if ((rc = call_encode_bf16(&m[0], p.a.ptr, cols_a, p.a.rows, p.a.ld, z_a, p.a.stride, kBK, box_a))) return rc;
        if ((rc = call_encode_bf16(&m[1], p.b.ptr, cols_b, p.b.rows, p.b.ld, parts, p.b.stride, kBK, box_b))) return rc;
        m[2] = m[4] = m[0];
        m[3] = m[5] = m[1];
        const bool ragged = p.rows_on_k && p.offsets;  // lists may end inside a block
        if (ragged) {
            if ((rc = call_encode_bf16(&m[2], p.a.ptr, cols_a, p.a.rows * parts, p.a.ld, 0, 0, kBK, 1))) return rc;
            if ((rc = call_encode_bf16(&m[4], p.a.ptr, cols_a, p.a.rows, p.a.ld, z_a, p.a.stride, kBK, 16))) return rc;
            if ((rc = call_encode_bf16(&m[5], p.b.ptr, cols_b, p.b.rows, p.b.ld, parts, p.b.stride, kBK, 16))) return rc;
        }
        if (ragged || q.list) {
            if ((rc = call_encode_bf16(&m[3], p.b.ptr, cols_b, p.b.rows * parts, p.b.ld, 0, 0, kBK, 1))) return rc;
        }
    }
    const int64_t units = t.whole + (t.tiles - t.whole) * (t.halved ? 2 : t.split);
    cudaError_t e;
    auto with_bn = [&](auto f32) {
        constexpr bool F = decltype(f32)::value;
        switch (t.bn) {
            case 32: return launch<32, F>(m, q, units, c.sms, st);
            case 64: return launch<64, F>(m, q, units, c.sms, st);
            case 128: return launch<128, F>(m, q, units, c.sms, st);
            default: return launch<256, F>(m, q, units, c.sms, st);
        }
    };
    e = parts == 3 ? with_bn(std::true_type()) : with_bn(std::false_type());
    if (e != cudaSuccess) return call_fail_cuda(e, "tensor-core layer product");
    *launches += 1;
    if (t.split > 1) {
        auto sum = parts == 3 ? sum_slices_kernel<true> : sum_slices_kernel<false>;
        e = launch_kernel(true, sum, dim3(static_cast<unsigned>(t.tiles * (t.bn / kSumCols))), dim3(2 * kBI), 0, st, q,
                          t.bn, static_cast<int>(t.tiles));
        if (e != cudaSuccess) return call_fail_cuda(e, "sum of K slices");
        *launches += 1;
    }
    return 0;
}

}  // namespace pg
