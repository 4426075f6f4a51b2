// tile_mx4_matmul: out[m][n] = t_a t_b sum_k a[m][k] b[n][k] of two matrices in
// microscaled 4-bit floats, by the tensor instructions that apply the blocks' scales
// themselves and accumulate in fp32.
//
// A CTA computes tiles of 128 rows of one operand by BN rows of the other, over all of
// K or a slice of it.  Warp roles:
//   a producer thread: stages of 256 columns (128 bytes of codes a row) of both
//   operands by bulk tensor copies with the 128-byte swizzle, and the scale tiles that
//   go with them by 1-D bulk copies;
//   a tensor warp: copies a stage's scales into tensor memory, issues the stage's
//   products (64 columns each), and hands the stage back when they are done, all by an
//   elected lane of the whole warp (a lane chosen by its number issued at half the rate:
//   8192 x 16384 x 8192 673 us instead of 386);
//   four epilogue warps: a finished tile from tensor memory, scaled by t_a t_b.
// Each stage has scale columns of its own in tensor memory, so that new scales never
// meet products still under way.
//
// The rows of b are the instructions' 128 rows and those of a their columns, so that with few
// rows of a no product is spent on rows that are not there but up to the next of 16, 32, 64
// and 128, and the lanes of a warp store neighbours.  K is cut over the CTAs of a cluster
// until the device is full, and the CTAs add their parts through each other's shared
// memory, in the order of the slices.
//
// Bound by the start (2.6 us with one stage), the cluster's sum (1.3) and the latency of the
// stages' first loads; large ones by memory.  Blocks of 16, operands from device memory, us:
// 1 x 4096 x 4096 5.9 (1.6 TB/s), 1 x 16384 x 16384 26.6 (5.7 TB/s), 17 x 8191 x 8160 11.2, 128 x
// 8192 x 8192 13.9; without slices 8.5, 26.6, 14.5 and 16.0.
#include <algorithm>
#include <atomic>

#include "mbtile_elem.cuh"
#include "mbtile_layer.h"
#include "mbtile_mx4.cuh"
#include "mbtile_ptx.cuh"
#include "mbtile_tcgen05.cuh"

namespace mbt {
namespace {

constexpr int kMmThreads = 256;
constexpr int kMmRows = 128;              // of the instructions' first operand
constexpr int kMmStep = 256;              // columns of K per stage
constexpr int kMmMostStages = 8;
constexpr int kMmTmem = 512;              // columns
struct Mx4MatArgs {
    const uint8_t *sr, *sc;    // scales of the rows' and of the columns' operand
    const float *ta, *tb;
    void *out;
    int64_t R, C, K, ld_out;   // rows and columns of the tiles' matrix
    int64_t scale_tiles;       // across K
    int32_t steps;
    int32_t tiles_r, tiles_c;
    int32_t split;             // CTAs of a cluster, each a slice of K
    int32_t stages, accs;      // in shared memory, in tensor memory
    int32_t tmem;              // columns of tensor memory
    int32_t odt;
    int32_t vec;               // rows of out are whole aligned 16-byte chunks
    int32_t *status;
};

template <int BN, int BLOCK>
struct MmShape {
    static constexpr int kTiles = kMmStep / BLOCK / 4;        // scale tiles of 128 rows per stage
    static constexpr int kRowBytes = kMmRows * kBoxRowBytes;
    static constexpr int kColBytes = BN * kBoxRowBytes;
    static constexpr int kScaleBytes = kTiles * 512;
    static constexpr int kStage = kRowBytes + kColBytes + kScaleBytes * 2;
    static constexpr int kScaleCols = kTiles * 4 * 2;   // tensor memory of a stage's scales
    static constexpr int kAcc = BN < 32 ? 32 : BN;
    // A cluster's parts of this CTA's rows; a row's columns, and 16 bytes that spread the rows
    // over the banks.
    static constexpr int kRecvRow = BN * 4 + 16;
    static constexpr int kRecv = kRecvRow * kMmRows;
    static_assert(kStage % kSwizzleAtomBytes == 0);
    // Stages within `bytes` of shared memory, beside accs accumulators in tensor memory.
    static int stages(int bytes, int accs) {
        return std::min({bytes / kStage, (kMmTmem - accs * kAcc) / kScaleCols, kMmMostStages});
    }
};

// Tiles in groups of up to 16 down the rows, so that CTAs side by side share both operands.
__device__ __forceinline__ void tile_at(const Mx4MatArgs &a, int t, int *r, int *c) {
    const int per = 16 * a.tiles_c, g = t / per, first = g * 16, rows = min(16, a.tiles_r - first), left = t - g * per;
    *c = left / rows;
    *r = first + left - *c * rows;
}

// wait_bounded() by a whole warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtl &w) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity) || wait_bounded(bar, parity, w, true));
}

struct MmShared {
    uint64_t full[kMmMostStages], empty[kMmMostStages], acc_full[2], acc_empty[2], drain;
    uint32_t tmem;
    int abort_flag;
};

template <int BN, int BLOCK>
__global__ void __launch_bounds__(kMmThreads, 1)
    mbt_mx4_matmul_kernel(const __grid_constant__ CUtensorMap rows_map, const __grid_constant__ CUtensorMap cols_map,
                          const __grid_constant__ Mx4MatArgs a) {
    using S = MmShape<BN, BLOCK>;
    extern __shared__ unsigned char dyn_smem[];
    __shared__ __align__(8) MmShared sh;
    const uint32_t base = (smem_u32(dyn_smem) + kSwizzleAtomBytes - 1) & ~static_cast<uint32_t>(kSwizzleAtomBytes - 1);
    const int warp = static_cast<int>(warp_value(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    // This CTA is there, and its memory may be stored to: see the epilogue.  A CTA waits in the
    // allocation until what else its SM runs frees enough tensor memory.  No CTA waits for
    // another of its cluster between that and its own tensor memory's release but for this arrival
    // before it: two clusters that each held what a CTA of the other needs would wait for ever.
    if (a.split > 1) cluster_arrive();
    if (warp == 2) tmem_alloc<1>(smem_u32(&sh.tmem), a.tmem);
    if (warp == 1 && elect_one()) {
        prefetch_map(&rows_map);
        prefetch_map(&cols_map);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&sh.acc_full[b]), 1);
            mbar_init(smem_u32(&sh.acc_empty[b]), 4);
        }
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort_flag = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // the next kernel of the stream may be set up from now on; it waits for this one's end itself
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t tmem = warp_value(sh.tmem);
    const WaitCtl w{kDefaultWaitBudgetNs, &sh.abort_flag, a.status};
    const int rank = a.split > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int first_tile = a.split > 1 ? static_cast<int>(blockIdx.x) / a.split : static_cast<int>(blockIdx.x);
    const int stride = a.split > 1 ? 0x40000000 : static_cast<int>(gridDim.x);   // (a cluster has one tile)
    const int tiles = a.tiles_r * a.tiles_c;
    const int k0 = static_cast<int>(static_cast<int64_t>(a.steps) * rank / a.split);
    const int k1 = static_cast<int>(static_cast<int64_t>(a.steps) * (rank + 1) / a.split);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    bool in_epilogue = false;                // this thread has waited for the cluster's beginning
    auto fail = [&](int role, uint32_t stage, uint32_t parity) {
        report_timeout(w, role, stage, parity);
        *w.abort = 1;
    };
    if (warp == 0 && lane == 0) {
        uint32_t stage = 0, phase = 1;
        bool alive = true;
        for (int t = first_tile; t < tiles && alive; t += stride) {
            int tr, tc;
            tile_at(a, t, &tr, &tc);
            for (int k = k0; k < k1; ++k) {
                const uint32_t full = smem_u32(&sh.full[stage]);
                if (!wait_bounded(smem_u32(&sh.empty[stage]), phase, w, true)) {
                    fail(0, stage, phase);
                    alive = false;
                    break;
                }
                const uint32_t at = base + stage * S::kStage, sr = at + S::kRowBytes + S::kColBytes;
                const int64_t tile = static_cast<int64_t>(k) * S::kTiles;
                const uint32_t bytes = 512u * static_cast<uint32_t>(min(static_cast<int64_t>(S::kTiles), a.scale_tiles - tile));
                mbar_arrive_expect_tx(full, S::kRowBytes + S::kColBytes + bytes * 2);
                tma_load_2d(at, &rows_map, k * kBoxRowBytes, tr * kMmRows, full);
                tma_load_2d(at + S::kRowBytes, &cols_map, k * kBoxRowBytes, tc * BN, full);
                bulk_load_1d(sr, a.sr + (tr * a.scale_tiles + tile) * 512, bytes, full);
                bulk_load_1d(sr + S::kScaleBytes, a.sc + (tc * a.scale_tiles + tile) * 512, bytes, full);
                if (++stage == static_cast<uint32_t>(a.stages)) stage = 0, phase ^= 1;
            }
        }
    } else if (warp == 1) {
        constexpr uint32_t idesc = mx4_idesc<BLOCK>(kMmRows, BN);
        uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 1;
        bool alive = true;
        for (int t = first_tile; t < tiles && alive; t += stride) {
            if (!warp_wait(smem_u32(&sh.acc_empty[acc]), acc_phase, w)) {
                if (lane == 0) fail(2, acc, acc_phase);
                alive = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + acc * S::kAcc;
            for (int k = k0; k < k1; ++k) {
                if (!warp_wait(smem_u32(&sh.full[stage]), phase, w)) {
                    if (lane == 0) fail(1, stage, phase);
                    alive = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = base + stage * S::kStage, sr = at + S::kRowBytes + S::kColBytes;
                const uint32_t scols = tmem + a.accs * S::kAcc + stage * S::kScaleCols;
                const uint32_t ccols = scols + S::kTiles * 4;
                const int left = static_cast<int>(min(static_cast<int64_t>(4), (a.K - static_cast<int64_t>(k) * kMmStep + 63) / 64));
                const uint64_t da = desc_swizzled(at), db = desc_swizzled(at + S::kRowBytes);
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < S::kTiles; ++s) {
                        if (4 * s >= left * S::kTiles) break;            // (no scales there)
                        tmem_copy_scales<1>(scols + 4 * s, desc_rows16(sr + 512 * s));
                        tmem_copy_scales<1>(ccols + 4 * s, desc_rows16(sr + S::kScaleBytes + 512 * s));
                    }
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        if (m >= left) break;
                        const int s = m * S::kTiles / 4;                     // the product's scale tile
                        const uint32_t id = BLOCK == 32 ? (m & 1) * 2 : 0;   // the first of the bytes in a scale column
                        mma_mx4<1, BLOCK>(d, da + 2 * m, db + 2 * m, idesc | id << 4 | id << 29, scols + 4 * s,
                                          ccols + 4 * s, k > k0 || m > 0);
                    }
                    tc_commit(smem_u32(&sh.empty[stage]));
                }
                __syncwarp();
                if (++stage == static_cast<uint32_t>(a.stages)) stage = 0, phase ^= 1;
            }
            if (!alive) break;
            if (elect_one()) tc_commit(smem_u32(&sh.acc_full[acc]));
            __syncwarp();
            if (++acc == static_cast<uint32_t>(a.accs)) acc = 0, acc_phase ^= 1;
        }
        if (!alive) {                        // what has been issued ends before tensor memory is freed
            if (elect_one()) tc_commit(smem_u32(&sh.drain));
            __syncwarp();
            wait_bounded(smem_u32(&sh.drain), 0, w, false);
        }
    } else if (warp >= 4) {
        const int quarter = warp & 3;
        float alpha = a.ta ? *a.ta : 1.f;
        if (a.tb) alpha *= *a.tb;
        uint32_t acc = 0, phase = 0;
        for (int t = first_tile; t < tiles; t += stride) {
            int tr, tc;
            tile_at(a, t, &tr, &tc);
            if (!warp_wait(smem_u32(&sh.acc_full[acc]), phase, w)) {
                if (lane == 0) fail(3, acc, phase);
                break;
            }
            tc_fence_after();
            const uint32_t from = tmem + acc * S::kAcc + (static_cast<uint32_t>(quarter * 32) << 16);
            const int r = quarter * 32 + lane;
            const int64_t row = static_cast<int64_t>(tr) * kMmRows + r, col0 = static_cast<int64_t>(tc) * BN;
            const int cols = static_cast<int>(min(static_cast<int64_t>(BN), a.C - col0));
            const int owned = kMmRows / a.split;
            uint32_t owner = 0;
            if (a.split > 1) {
                cluster_wait();              // every CTA of the cluster has begun
                in_epilogue = true;
                owner = cluster_address(base + a.stages * S::kStage + (rank * owned + r % owned) * S::kRecvRow, r / owned);
            }
#pragma unroll 2
            for (int c = 0; c < BN; c += 16) {
                if (c >= cols) break;
                float f[16];
                __syncwarp();
                tmem_load16(from + c, f);
                if (a.split > 1) {   // the slice's sums, to the CTA that adds the row's
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        if (c + e < cols) cluster_store(owner + (c + e) * 4, make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]));
                } else if (row < a.R) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] *= alpha;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (c + e < cols) store_any(a.out, a.odt, (col0 + c + e) * a.ld_out + row, f[e]);
                }
            }
            __syncwarp();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sh.acc_empty[acc]));
            if (++acc == static_cast<uint32_t>(a.accs)) acc = 0, phase ^= 1;
        }
    }
    __syncwarp();
    bool freed = false;
    if (a.split > 1) {
        // A CTA adds rows of its own from every CTA's part, in the slices' order.  (Parts are
        // stored into the memory of the CTA that adds them, apart from its stages, which it may
        // still use: one barrier, after which no CTA needs another's memory.)
        if (!in_epilogue) cluster_wait();
        cluster_arrive();
        if (warp == 2 && warp_wait(smem_u32(&sh.acc_empty[0]), 0, w)) {   // (its tile has been read)
            tc_fence_after();
            tmem_free<1>(tmem, a.tmem);
            freed = true;
        }
        cluster_wait();
        float alpha = a.ta ? *a.ta : 1.f;
        if (a.tb) alpha *= *a.tb;
        int tr, tc;
        tile_at(a, first_tile, &tr, &tc);
        const int owned = kMmRows / a.split;
        const int64_t row0 = static_cast<int64_t>(tr) * kMmRows + rank * owned, col0 = static_cast<int64_t>(tc) * BN;
        const int cols = static_cast<int>(min(static_cast<int64_t>(BN), a.C - col0));
        const int r = threadIdx.x & (owned - 1), at_once = kMmThreads / owned * 4;   // (owned: a power of two)
        const uint32_t recv = base + a.stages * S::kStage + r * S::kRecvRow;
        for (int c = threadIdx.x / owned * 4; c < cols; c += at_once) {
            float4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (q < a.split) {
                    const uint4 u = lds128(recv + q * owned * S::kRecvRow + c * 4);
                    v[q] = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
                }
            float4 sum = v[0];
#pragma unroll
            for (int q = 1; q < 8; ++q)
                if (q < a.split) sum.x += v[q].x, sum.y += v[q].y, sum.z += v[q].z, sum.w += v[q].w;
            const float f[4] = {sum.x * alpha, sum.y * alpha, sum.z * alpha, sum.w * alpha};
            if (row0 + r < a.R)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < cols) store_any(a.out, a.odt, (col0 + c + e) * a.ld_out + row0 + r, f[e]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sh.abort_flag)   // copies under way land before the CTA leaves
        for (int s = 0; s < a.stages; ++s)
            for (uint32_t p = 0; p < 2; ++p) wait_bounded(smem_u32(&sh.full[s]), p, w, false);
    __syncthreads();
    tc_fence_after();
    if (warp == 2 && !freed) tmem_free<1>(tmem, a.tmem);
}

// ---------------------------------------------------------------------------
// Many rows: a pair of CTAs on 256 x 256
// ---------------------------------------------------------------------------
// The two CTAs of a cluster hold 128 rows each of both operands, and the pair's tensor
// instructions read both: a byte of shared memory filled from L2 serves twice the products
// of a 128 x 128 tile, whose rate the L2's was.  Each CTA accumulates its 128 rows by 256
// columns and needs the scales of its rows and of all columns.  The first CTA's tensor
// thread issues for both; copies of either CTA count on its barriers.
//
// 8192 x 16384 x 8192 by 16 takes 374 us in use, 5.9 PFLOP/s, with the clock held at 1.8 GHz by
// the power cap (346 before the cap, with the tensor pipe busy for 67 % of it: the copies alone
// 316 us, 55 of the 64 bytes a cycle that an SM takes in, the products alone 230).  1024 x 8192 x
// 8192 29.5 us, 4.7 PFLOP/s.
//
// Two accumulators of 256 columns would leave no tensor memory for scales: there is one,
// and eight epilogue warps take all of it into registers before they convert and store,
// so that the next tile's products wait for that alone.
constexpr int kPairThreads = 384;
constexpr int kPairCols = 256;

template <int BLOCK>
struct PairShape {
    static constexpr int kTiles = kMmStep / BLOCK / 4;        // scale tiles of 128 rows per stage
    static constexpr int kOperand = kMmRows * kBoxRowBytes;   // of a CTA's part of either operand
    static constexpr int kScaleBytes = kTiles * 512;
    static constexpr int kStage = 2 * kOperand + 3 * kScaleBytes;
    static constexpr int kStageStride = (kStage + kSwizzleAtomBytes - 1) / kSwizzleAtomBytes * kSwizzleAtomBytes;
    static constexpr int kScaleCols = kTiles * 4 * 3;
    static constexpr int kStages = 5;
    static constexpr int kOutBox = 32 * kBoxRowBytes;         // 32 rows of an epilogue warp, 128 bytes of each
    // (At least: the CTAs of a pair wait for each other with tensor memory in hand, so an SM that
    // holds one is to hold no other CTA that might do the same.)
    static constexpr int kLeast = 225 * 1024;
    static constexpr int kNeeds = kStages * kStageStride + 8 * kOutBox + kSwizzleAtomBytes;
    static constexpr int kSmem = kNeeds > kLeast ? kNeeds : kLeast;
    static_assert(kPairCols + kStages * kScaleCols <= kMmTmem && kSmem <= 226 * 1024);
};

struct PairShared {
    uint64_t full[kMmMostStages], empty[kMmMostStages], acc_full, acc_empty, drain;
    uint32_t tmem;
    int abort_flag;
};

// An element of 2 or 4 bytes from shared to global memory.
template <int ES>
__device__ __forceinline__ void copy_staged(void *to, uint32_t from) {
    if constexpr (ES == 2) {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(from) : "memory");
        *static_cast<uint16_t *>(to) = v;
    } else {
        uint32_t v;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(from) : "memory");
        *static_cast<uint32_t *>(to) = v;
    }
}

// A warp's 32 rows x 128 columns of results to out, a box of 128 bytes of each row at a time.
template <int DT>
__device__ __forceinline__ void put_box(const uint32_t (&acc)[kPairCols / 2], float alpha, uint32_t staged,
                                        const CUtensorMap *map, void *out, int64_t ld_out, int64_t row0, int64_t col0, int64_t R,
                                        int64_t C, int lane) {
    constexpr int V = Elem<DT>::kVec, es = 16 / V, kBox = kBoxRowBytes / es;   // columns of a box
#pragma unroll
    for (int b = 0; b < kPairCols / 2; b += kBox) {
        if (row0 >= R || col0 + b >= C) break;
        if (lane == 0) bulk_wait_read_all();                     // the box before this one
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = __uint_as_float(acc[b + j * V + e]) * alpha;
            const uint4 v = pack<DT>(f);
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(staged + lane * kBoxRowBytes + ((j ^ (lane & 7)) << 4)),
                         "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                         : "memory");
        }
        if (col0 + b + kBox > C) {           // (a bulk copy would write whole 16 bytes at the rows' end)
            if (row0 + lane < R)
#pragma unroll 1
                for (int e = 0; e < static_cast<int>(C - col0 - b); ++e)
                    copy_staged<es>(static_cast<char *>(out) + ((row0 + lane) * ld_out + col0 + b + e) * es,
                                    staged + lane * kBoxRowBytes + (((e / V) ^ (lane & 7)) << 4) + e % V * es);
            __syncwarp();
            break;
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(map, staged, static_cast<int32_t>((col0 + b) * es), static_cast<int32_t>(row0));
            bulk_commit_group();
        }
    }
}

template <int BLOCK>
__global__ void __launch_bounds__(kPairThreads, 1)
    mbt_mx4_pair_kernel(const __grid_constant__ CUtensorMap rows_map, const __grid_constant__ CUtensorMap cols_map,
                        const __grid_constant__ CUtensorMap row_scales, const __grid_constant__ CUtensorMap col_scales,
                        const __grid_constant__ CUtensorMap out_map, const __grid_constant__ Mx4MatArgs a) {
    using S = PairShape<BLOCK>;
    extern __shared__ unsigned char dyn_smem[];
    __shared__ __align__(8) PairShared sh;
    const uint32_t base = (smem_u32(dyn_smem) + kSwizzleAtomBytes - 1) & ~static_cast<uint32_t>(kSwizzleAtomBytes - 1);
    const int warp = static_cast<int>(warp_value(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (warp == 2) tmem_alloc<2>(smem_u32(&sh.tmem), kMmTmem);
    if (warp == 1 && elect_one()) {
        prefetch_map(&rows_map);
        prefetch_map(&cols_map);
        prefetch_map(&row_scales);
        prefetch_map(&col_scales);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(smem_u32(&sh.full[s]), 1);
            mbar_init(smem_u32(&sh.empty[s]), 1);
        }
        mbar_init(smem_u32(&sh.acc_full), 1);
        mbar_init(smem_u32(&sh.acc_empty), 16);
        mbar_init(smem_u32(&sh.drain), 1);
        sh.abort_flag = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();                          // both CTAs' barriers are there
    tc_fence_after();
    asm volatile("griddepcontrol.launch_dependents;");       // (see above)
    const uint32_t tmem = warp_value(sh.tmem);
    const WaitCtl w{kDefaultWaitBudgetNs, &sh.abort_flag, a.status};
    const int first_tile = static_cast<int>(blockIdx.x >> 1), stride = static_cast<int>(gridDim.x >> 1);
    const int tiles = a.tiles_r * a.tiles_c;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    auto fail = [&](int role, uint32_t stage, uint32_t parity) {
        report_timeout(w, role, stage, parity);
        *w.abort = 1;
    };
    if (warp == 0 && lane == 0) {
        uint32_t stage = 0, phase = 1;
        bool alive = true;
        for (int t = first_tile; t < tiles && alive; t += stride) {
            int tr, tc;
            tile_at(a, t, &tr, &tc);
            for (int k = 0; k < a.steps; ++k) {
                if (!wait_bounded(smem_u32(&sh.empty[stage]), phase, w, true)) {
                    fail(0, stage, phase);
                    alive = false;
                    break;
                }
                const uint32_t full = cluster_address(smem_u32(&sh.full[stage]), 0);
                const uint32_t at = base + stage * S::kStageStride, sc = at + 2 * S::kOperand;
                // (boxes past the matrix's end are filled with zeros and count in full)
                if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh.full[stage]), 2 * S::kStage);
                tma_load_2d_pair(at, &rows_map, k * kBoxRowBytes, (2 * tr + static_cast<int>(rank)) * kMmRows, full);
                tma_load_2d_pair(at + S::kOperand, &cols_map, k * kBoxRowBytes, (2 * tc + static_cast<int>(rank)) * kMmRows,
                                 full);
                tma_load_3d_pair(sc, &row_scales, 0, k * S::kTiles, 2 * tr + static_cast<int>(rank), full);
                tma_load_3d_pair(sc + S::kScaleBytes, &col_scales, 0, k * S::kTiles, 2 * tc, full);
                tma_load_3d_pair(sc + 2 * S::kScaleBytes, &col_scales, 0, k * S::kTiles, 2 * tc + 1, full);
                if (++stage == S::kStages) stage = 0, phase ^= 1;
            }
        }
    } else if (warp == 1 && rank == 0) {
        constexpr uint32_t idesc = mx4_idesc<BLOCK>(2 * kMmRows, kPairCols);
        uint32_t stage = 0, phase = 0, acc_phase = 1;
        bool alive = true;
        for (int t = first_tile; t < tiles && alive; t += stride) {
            if (!warp_wait(smem_u32(&sh.acc_empty), acc_phase, w)) {
                if (lane == 0) fail(2, 0, acc_phase);
                alive = false;
                break;
            }
            acc_phase ^= 1;
            tc_fence_after();
            for (int k = 0; k < a.steps; ++k) {
                if (!warp_wait(smem_u32(&sh.full[stage]), phase, w)) {
                    if (lane == 0) fail(1, stage, phase);
                    alive = false;
                    break;
                }
                tc_fence_after();
                const uint32_t at = base + stage * S::kStageStride, sc = at + 2 * S::kOperand;
                const uint32_t scols = tmem + kPairCols + stage * S::kScaleCols, ccols = scols + S::kTiles * 4;
                const int left = static_cast<int>(min(static_cast<int64_t>(4), (a.K - static_cast<int64_t>(k) * kMmStep + 63) / 64));
                const uint64_t da = desc_swizzled(at), db = desc_swizzled(at + S::kOperand);
                if (elect_one()) {
#pragma unroll
                    for (int s = 0; s < S::kTiles; ++s) {
                        tmem_copy_scales<2>(scols + 4 * s, desc_rows16(sc + 512 * s));
                        tmem_copy_scales<2>(ccols + 8 * s, desc_rows16(sc + S::kScaleBytes + 512 * s));
                        tmem_copy_scales<2>(ccols + 8 * s + 4, desc_rows16(sc + 2 * S::kScaleBytes + 512 * s));
                    }
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        if (m >= left) break;
                        const int s = m * S::kTiles / 4;                     // the product's scale tile
                        const uint32_t id = BLOCK == 32 ? (m & 1) * 2 : 0;   // the first of the bytes in a scale column
                        mma_mx4<2, BLOCK>(tmem, da + 2 * m, db + 2 * m, idesc | id << 4 | id << 29, scols + 4 * s,
                                          ccols + 8 * s, k > 0 || m > 0);
                    }
                    tc_commit_pair(smem_u32(&sh.empty[stage]), 3);
                }
                __syncwarp();
                if (++stage == S::kStages) stage = 0, phase ^= 1;
            }
            if (!alive) break;
            if (elect_one()) tc_commit_pair(smem_u32(&sh.acc_full), 3);
            __syncwarp();
        }
        if (!alive) {                        // what has been issued ends before tensor memory is freed
            if (elect_one()) tc_commit_pair(smem_u32(&sh.drain), 1);
            __syncwarp();
            wait_bounded(smem_u32(&sh.drain), 0, w, false);
        }
    } else if (warp >= 4) {
        const int quarter = warp & 3, half = (warp - 4) >> 2;
        float alpha = a.ta ? *a.ta : 1.f;
        if (a.tb) alpha *= *a.tb;
        const uint32_t acc_empty = cluster_address(smem_u32(&sh.acc_empty), 0);
        constexpr int kCols = kPairCols / 2;                     // of a warp
        const uint32_t staged = base + S::kStages * S::kStageStride + (warp - 4) * S::kOutBox;
        uint32_t phase = 0;
        for (int t = first_tile; t < tiles; t += stride) {
            int tr, tc;
            tile_at(a, t, &tr, &tc);
            if (!warp_wait(smem_u32(&sh.acc_full), phase, w)) {
                if (lane == 0) fail(3, 0, phase);
                break;
            }
            phase ^= 1;
            tc_fence_after();
            const uint32_t from = tmem + half * kCols + (static_cast<uint32_t>(quarter * 32) << 16);
            const int64_t row0 = (static_cast<int64_t>(tr) * 2 + rank) * kMmRows + quarter * 32, row = row0 + lane;
            const int64_t col0 = static_cast<int64_t>(tc) * kPairCols + half * kCols;
            const int cols = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(kCols), a.C - col0)));
            uint32_t acc[kCols];
            __syncwarp();
            tmem_load128(from, acc);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) cluster_arrive_at(acc_empty);
            if (!a.vec) {
                if (row < a.R)
#pragma unroll
                    for (int c = 0; c < kCols; ++c)
                        if (c < cols) store_any(a.out, a.odt, row * a.ld_out + col0 + c, __uint_as_float(acc[c]) * alpha);
                continue;
            }
            // By way of shared memory, in the swizzle's order, and bulk tensor copies of 128
            // bytes of 32 rows: 16 bytes a lane and row straight from the registers, 32 rows an
            // instruction, took 85 us of 414.
            if (a.odt == MBT_F32)
                put_box<MBT_F32>(acc, alpha, staged, &out_map, a.out, a.ld_out, row0, col0, a.R, a.C, lane);
            else if (a.odt == MBT_BF16)
                put_box<MBT_BF16>(acc, alpha, staged, &out_map, a.out, a.ld_out, row0, col0, a.R, a.C, lane);
            else
                put_box<MBT_F16>(acc, alpha, staged, &out_map, a.out, a.ld_out, row0, col0, a.R, a.C, lane);
        }
        if (lane == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && rank == 0 && sh.abort_flag)   // copies under way land before the CTAs leave
        for (int s = 0; s < S::kStages; ++s)
            for (uint32_t p = 0; p < 2; ++p) wait_bounded(smem_u32(&sh.full[s]), p, w, false);
    __syncthreads();
    cluster_sync();                          // nor does a CTA leave while the other may still signal it
    tc_fence_after();
    if (warp == 2) tmem_free<2>(tmem, kMmTmem);
}

template <int BLOCK>
int launch_pair(const uint8_t *rows, int64_t ld_rows, const uint8_t *cols, int64_t ld_cols, Mx4MatArgs a, int sms,
                cudaStream_t stream) {
    using S = PairShape<BLOCK>;
    static std::atomic<bool> raised[64];   // per device: the kernel's shared-memory limit is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MBT_ERR_CUDA;
    if (dev >= 64 || !raised[dev].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(mbt_mx4_pair_kernel<BLOCK>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) !=
            cudaSuccess)
            return MBT_ERR_CUDA;
        if (dev < 64) raised[dev].store(true, std::memory_order_relaxed);
    }
    alignas(64) CUtensorMap maps[5] = {};
    int rc = encode_bytes_map(&maps[0], rows, a.R, a.K / 2, ld_rows, kMmRows);
    if (rc == MBT_OK) rc = encode_bytes_map(&maps[1], cols, a.C, a.K / 2, ld_cols, kMmRows);
    if (rc == MBT_OK) rc = encode_scales_map(&maps[2], a.sr, (a.R + 127) / 128, a.scale_tiles, S::kTiles);
    if (rc == MBT_OK) rc = encode_scales_map(&maps[3], a.sc, (a.C + 127) / 128, a.scale_tiles, S::kTiles);
    const int64_t es = a.odt == MBT_F32 ? 4 : 2;
    a.vec = a.vec && a.C * es <= 0x7fffffff;                  // (a map's coordinates are bytes, in 32 bits)
    if (rc == MBT_OK && a.vec) rc = encode_bytes_map(&maps[4], a.out, a.R, a.C * es, a.ld_out * es, 32);
    if (rc != MBT_OK) return rc;
    a.tiles_r = static_cast<int32_t>((a.R + 2 * kMmRows - 1) / (2 * kMmRows));
    a.tiles_c = static_cast<int32_t>((a.C + kPairCols - 1) / kPairCols);
    a.split = 1;
    const int64_t tiles = static_cast<int64_t>(a.tiles_r) * a.tiles_c;
    if (tiles > 0x3fffffff) return MBT_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(tiles, sms / 2)));
    cfg.blockDim = dim3(kPairThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mbt_mx4_pair_kernel<BLOCK>, maps[0], maps[1], maps[2], maps[3], maps[4], a) == cudaSuccess
               ? MBT_OK
               : MBT_ERR_CUDA;
}

__global__ void mbt_mx4_zero_kernel(void *out, int dtype, int64_t M, int64_t N, int64_t ld) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t e = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; e < M * N;
         e += static_cast<int64_t>(gridDim.x) * blockDim.x)
        store_any(out, dtype, e / N * ld + e % N, 0.f);
}

bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

constexpr int kMmSmem = 226 * 1024 - 1024;   // for stages and what a cluster's CTAs leave each other

template <int BN, int BLOCK>
int launch_matmul(const uint8_t *rows, int64_t ld_rows, const uint8_t *cols, int64_t ld_cols, Mx4MatArgs a, int sms,
                  cudaStream_t stream) {
    using S = MmShape<BN, BLOCK>;
    static std::atomic<bool> raised[64];   // per device: the kernel's shared-memory limit is set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MBT_ERR_CUDA;
    if (dev >= 64 || !raised[dev].load(std::memory_order_relaxed)) {
        if (cudaFuncSetAttribute(mbt_mx4_matmul_kernel<BN, BLOCK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMmSmem + kSwizzleAtomBytes) != cudaSuccess)
            return MBT_ERR_CUDA;
        if (dev < 64) raised[dev].store(true, std::memory_order_relaxed);
    }
    alignas(64) CUtensorMap rows_map, cols_map;
    int rc = encode_bytes_map(&rows_map, rows, a.R, a.K / 2, ld_rows, kMmRows);
    if (rc == MBT_OK) rc = encode_bytes_map(&cols_map, cols, a.C, a.K / 2, ld_cols, BN);
    if (rc != MBT_OK) return rc;
    a.tiles_r = static_cast<int32_t>((a.R + kMmRows - 1) / kMmRows);
    a.tiles_c = static_cast<int32_t>((a.C + BN - 1) / BN);
    const int64_t tiles = static_cast<int64_t>(a.tiles_r) * a.tiles_c;
    if (tiles > 0x3fffffff) return MBT_ERR_UNSUPPORTED;
    a.split = 1;
    while (a.split < 8 && tiles * a.split * 2 <= sms && a.split * 2 <= a.steps) a.split *= 2;
    // As many stages, accumulators and columns of tensor memory as a CTA has use for: what
    // is left lets the next kernel's CTAs set up while this one's finish.
    const int64_t ctas = a.split > 1 ? tiles * a.split : std::min<int64_t>(tiles, sms);
    const int64_t turns = a.split > 1 ? 1 : (tiles + ctas - 1) / ctas;
    const int recv = a.split > 1 ? S::kRecv : 0;
    a.accs = turns > 1 ? 2 : 1;
    a.stages = static_cast<int32_t>(std::min<int64_t>(S::stages(kMmSmem - recv, a.accs), turns * ((a.steps + a.split - 1) / a.split)));
    a.tmem = 64;
    while (a.tmem < a.accs * S::kAcc + a.stages * S::kScaleCols) a.tmem *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.stages * S::kStage + recv + kSwizzleAtomBytes);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.split);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, mbt_mx4_matmul_kernel<BN, BLOCK>, rows_map, cols_map, a) == cudaSuccess
               ? MBT_OK
               : MBT_ERR_CUDA;
}

// A wave of 128 x 128 tiles has the device's SMs to itself, cut along K if need be; more of
// them than that are slower than pairs (us, alone / by pairs): 256 x 4096 x 4096 9.8 / 10.7,
// 512 x 8192 x 8192 26.9 / 17.0, 1024 x 8192 x 512 10.1 / 8.5, 2048 x 8192 x 2048 25.8 / 22.1.
bool pair_pays(int64_t M, int64_t N, int sms) { return (M + 127) / 128 * ((N + 127) / 128) > sms; }

template <int BLOCK>
int matmul(const uint8_t *a_q, int64_t ld_a, const uint8_t *b_q, int64_t ld_b, const uint8_t *as, const uint8_t *bs,
           int64_t M, int64_t N, Mx4MatArgs a, int sms, cudaStream_t s) {
    if (M > 128 && pair_pays(M, N, sms)) {
        a.R = M, a.C = N, a.sr = as, a.sc = bs;
        return launch_pair<BLOCK>(a_q, ld_a, b_q, ld_b, a, sms, s);
    }
    a.R = N, a.C = M, a.sr = bs, a.sc = as;
    return M <= 16   ? launch_matmul<16, BLOCK>(b_q, ld_b, a_q, ld_a, a, sms, s)
           : M <= 32 ? launch_matmul<32, BLOCK>(b_q, ld_b, a_q, ld_a, a, sms, s)
           : M <= 64 ? launch_matmul<64, BLOCK>(b_q, ld_b, a_q, ld_a, a, sms, s)
                     : launch_matmul<128, BLOCK>(b_q, ld_b, a_q, ld_a, a, sms, s);
}

}  // namespace
}  // namespace mbt

extern "C" int tile_mx4_matmul(const uint8_t *a, const uint8_t *a_scales, const float *a_tensor_scale, const uint8_t *b,
                               const uint8_t *b_scales, const float *b_tensor_scale, void *out, int64_t M, int64_t N,
                               int64_t K, int64_t ld_a, int64_t ld_b, int64_t ld_out, int block, int out_dtype,
                               void *stream) {
    using namespace mbt;
    if (M < 0 || N < 0 || K < 0 || M > 0x7fffffff || N > 0x7fffffff || K > 0x7fffffff || out_dtype < MBT_F16 ||
        out_dtype > MBT_F32)
        return MBT_ERR_ARG;
    if ((block != 16 && block != 32) || K % 32 != 0) return MBT_ERR_UNSUPPORTED;
    if (block != 16 && (a_tensor_scale || b_tensor_scale)) return MBT_ERR_ARG;
    if (ld_a == 0) ld_a = K / 2;
    if (ld_b == 0) ld_b = K / 2;
    if (ld_out == 0) ld_out = N;
    if (ld_a < K / 2 || ld_b < K / 2 || ld_out < N || ld_a >= (1ll << 40) || ld_b >= (1ll << 40) || ld_out > (1ll << 40))
        return MBT_ERR_ARG;
    if (M == 0 || N == 0) return MBT_OK;
    if (!out || (K > 0 && (!a || !a_scales || !b || !b_scales))) return MBT_ERR_ARG;
    const uintptr_t es = out_dtype == MBT_F32 ? 4 : 2;
    if (!aligned(out, es) || !aligned(a, 16) || !aligned(b, 16) || !aligned(a_scales, 16) || !aligned(b_scales, 16) ||
        ld_a % 16 != 0 || ld_b % 16 != 0 || !aligned(a_tensor_scale, 4) || !aligned(b_tensor_scale, 4))
        return MBT_ERR_ALIGN;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (K == 0) {
        mbt_mx4_zero_kernel<<<1024, 256, 0, s>>>(out, out_dtype, M, N, ld_out);
        return cudaGetLastError() == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
    }
    int sms = 0, optin = 0;
    int rc = device_limits(&sms, &optin);
    if (rc != MBT_OK) return rc;
    Mx4MatArgs g{};
    rc = device_status_word(&g.status);
    if (rc != MBT_OK) return rc;
    g.ta = a_tensor_scale;
    g.tb = b_tensor_scale;
    g.out = out;
    g.K = K;
    g.ld_out = ld_out;
    g.scale_tiles = mx4_tiles(K, block);
    g.steps = static_cast<int32_t>((K + kMmStep - 1) / kMmStep);
    g.odt = out_dtype;
    g.vec = aligned(out, 16) && ld_out * static_cast<int64_t>(es) % 16 == 0;
    return block == 16 ? matmul<16>(a, ld_a, b, ld_b, a_scales, b_scales, M, N, g, sms, s)
                       : matmul<32>(a, ld_a, b, ld_b, a_scales, b_scales, M, N, g, sms, s);
}
