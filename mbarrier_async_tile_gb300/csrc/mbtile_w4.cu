// tile_w4_matvec: products of a few rows of activations with a matrix held in
// 4 bits, y[t, n] = sum_k x[t, k] (q[n, k] - z[n, k / g]) s[n, k / g].
//
// The matrix is read once and each of its elements used at most eight times:
// device memory bounds the large products, latency the small ones.
//
// A CTA takes 128 rows of q and a slice of K; a cluster of up to eight CTAs
// takes the slices of one row block and adds them, in rank order, through
// distributed shared memory.  Warp roles:
//   8 consumer warps, 16 rows each;
//   a producer thread: tiles of 128 rows x 256 columns (128 bytes) of q by bulk
//   tensor copies into a ring of 128-byte-swizzled stages;
//   2 staging warps: x and the scales in segments of 512 columns, converted
//   once per CTA, through a second ring.
//
// The products are m16n8k16 tensor instructions with 16 rows of q as A and
// eight rows of x as B.  (Tcgen05's smallest tile has 64 rows against 8 columns
// and takes both operands from shared memory or its own memory, where q would
// first have to be written back in 16 bits; here q goes from registers.)
// An A element is a 4-bit value left where it lies in a 16-bit half: bits 0..3
// are the fp16 subnormal q 2^-24 and bits 4..7 are q 2^-20, both exact, so
// extracting eight values costs four ANDs and a shift.  B's elements for bits
// 4..7 are divided by 16 beforehand.  Which k goes where in the instruction is
// free as long as A and B agree: a 16-byte chunk of a row (32 columns) is read
// by ldmatrix as if it held 16-bit elements, which gives the lane of column
// pair j the bytes 4j..4j+3, columns 8j..8j+7; nibbles i and i + 4 share a half
// pair.
//
// x is scaled by a power of two per row and group (16-bit inputs of any range
// then fit fp16: values below 2^-29 of the group's largest lose bits, less than
// fp32 sums do), and each group's product is taken back in fp32:
//   acc += s 2^24 (p 2^-e - z 2^-24 sum x).
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "mbtile_elem.cuh"
#include "mbtile_layer.h"
#include "mbtile_ptx.cuh"

namespace mbt {
namespace {

constexpr int kW4Rows = 128;              // rows of q per CTA
constexpr int kW4Step = 256;              // columns per stage of q
constexpr int kW4Seg = 512;               // columns per segment of x
constexpr int kW4Consumers = 8;           // warps
constexpr int kW4Threads = 32 * (kW4Consumers + 1) + 64;
constexpr int kW4StageBytes = kW4Rows * kW4Step / 2;
constexpr int kW4Segs = 2;                // segments of x staged ahead
constexpr int kW4Tokens = 8;
constexpr int kW4MaxSlices = 8;           // portable cluster size
constexpr int kW4MaxSmem = 104 * 1024;    // dynamic; two CTAs fit an SM

struct W4Args {
    const void *x;
    const void *s;
    const uint8_t *z;
    const float *xs;
    void *out;
    int64_t T, N, K, ld_x, ld_out;
    int64_t groups, x_groups;   // scales of a row of q, of a row of x
    int32_t xdt, sdt, odt;
    int32_t x_row_scale;        // e4m3: a scale per row of x, else per 128 columns
    int32_t slices;             // CTAs of a cluster, along K
    int32_t vec_scales;         // a segment's scales of a row are aligned vectors
    int32_t vec_zeros;
    int32_t vec_x;              // eight columns of x are one aligned vector
    int32_t *status;
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct W4Rings {
    uint32_t q, x;              // shared-memory addresses of the rings
    uint32_t x_bytes;           // x's part of a segment buffer
    uint32_t seg_bytes;         // x, then {2^-e, 2^-24 sum x} per group and token, then
                                // {s 2^24, z} per group and row of q
    uint32_t full_q, empty_q, full_x, empty_x;
};

template <int G>
struct W4Seg {
    static constexpr int kGroups = kW4Seg / G;
    static constexpr int kMeta = kGroups * kW4Tokens * 8;
    static constexpr int kScales = kGroups * kW4Rows * 8;
    // Stages of q: what is left of half an SM's shared memory beside the two
    // segments (of small groups there are more scales).
    static constexpr int kStages = G == 32 ? 3 : 4;
};

// Rows r and r + 8 of a warp's 16 are neighbours, so one 16-byte read gives a
// consumer lane both of its rows.
__device__ __forceinline__ int scale_slot(int row) {
    return (row & ~15) | (row & 7) << 1 | (row >> 3 & 1);
}

// A staging thread's two rows of the scales of segment `seg`.
template <int G, bool S32>
__device__ __forceinline__ void stage_scales(const W4Args &a, int64_t seg, int64_t row0, int u,
                                             uint32_t dst) {
    constexpr int kGroups = kW4Seg / G;
    constexpr int kWords = S32 ? kGroups : kGroups / 2;
    const int64_t g0 = seg * kGroups;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int local = u + 64 * h;
        const int64_t row = row0 + local;
        uint32_t w[kWords] = {};
        uint32_t z[(kGroups + 3) / 4];
#pragma unroll
        for (int i = 0; i < (kGroups + 3) / 4; ++i) z[i] = 0x08080808u;
        if (row < a.N) {
            const int64_t at = row * a.groups + g0;
            const char *s = static_cast<const char *>(a.s) + at * (S32 ? 4 : 2);
            if (a.vec_scales && g0 + kGroups <= a.groups) {
                if constexpr (kWords == 2) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(s));
                    w[0] = v.x, w[1] = v.y;
                } else {
#pragma unroll
                    for (int i = 0; i < kWords / 4; ++i) {
                        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(s) + i);
                        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    if (g0 + i >= a.groups) continue;
                    if constexpr (S32)
                        w[i] = __ldg(reinterpret_cast<const uint32_t *>(s) + i);
                    else
                        w[i / 2] |=
                            static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(s) + i))
                            << (16 * (i & 1));
                }
            }
            if (a.z) {
                if (a.vec_zeros && g0 + kGroups <= a.groups) {
#pragma unroll
                    for (int i = 0; i < kGroups / 4; ++i)
                        z[i] = __ldg(reinterpret_cast<const uint32_t *>(a.z + at) + i);
                } else {
#pragma unroll
                    for (int i = 0; i < kGroups; ++i) {
                        if (i % 4 == 0) z[i / 4] = 0;
                        if (g0 + i < a.groups)
                            z[i / 4] |= static_cast<uint32_t>(__ldg(a.z + at + i)) << (8 * (i % 4));
                    }
                }
            }
        }
        const uint32_t slot = dst + 8u * static_cast<uint32_t>(scale_slot(local));
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            float v;
            if constexpr (S32) {
                v = __uint_as_float(w[i]);
            } else {
                const uint32_t b = w[i / 2] >> (16 * (i & 1));
                v = a.sdt == MBT_BF16 ? __uint_as_float(b << 16) : Elem<MBT_F16>::widen2(b).x;
            }
            const float zero = static_cast<float>(z[i / 4] >> (8 * (i % 4)) & 0xffu);
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(slot + i * (8u * kW4Rows)),
                         "f"(v * 16777216.f), "f"(zero)
                         : "memory");
        }
    }
}

// A staging warp's half of segment `seg`: 8 columns a lane, every row of x.
template <int G>
__device__ __forceinline__ void stage_x(const W4Args &a, int64_t seg, int64_t t0, int tokens, int u,
                                        uint32_t xbuf, uint32_t meta) {
    const int64_t k = seg * kW4Seg + 8 * u;
    const bool in = k < a.K;
    uint4 raw[kW4Tokens];
#pragma unroll
    for (int t = 0; t < kW4Tokens; ++t) {
        raw[t] = make_uint4(0, 0, 0, 0);
        if (t >= tokens || !in) continue;
        const int64_t at = (t0 + t) * a.ld_x + k;
        if (a.xdt == MBT_E4M3) {
            const uint8_t *p = static_cast<const uint8_t *>(a.x) + at;
            uint2 v;
            if (a.vec_x) {
                v = __ldg(reinterpret_cast<const uint2 *>(p));
            } else {
                v = make_uint2(0, 0);
                for (int i = 0; i < 4; ++i) {
                    v.x |= static_cast<uint32_t>(p[i]) << (8 * i);
                    v.y |= static_cast<uint32_t>(p[4 + i]) << (8 * i);
                }
            }
            raw[t].x = v.x;
            raw[t].y = v.y;
        } else {
            const uint16_t *p = static_cast<const uint16_t *>(a.x) + at;
            if (a.vec_x) {
                raw[t] = __ldg(reinterpret_cast<const uint4 *>(p));
            } else {
                raw[t].x = p[0] | static_cast<uint32_t>(p[1]) << 16;
                raw[t].y = p[2] | static_cast<uint32_t>(p[3]) << 16;
                raw[t].z = p[4] | static_cast<uint32_t>(p[5]) << 16;
                raw[t].w = p[6] | static_cast<uint32_t>(p[7]) << 16;
            }
        }
    }
#pragma unroll
    for (int t = 0; t < kW4Tokens; ++t) {
        if (t >= tokens) break;
        float f[8];
        float factor = 1.f;
        if (a.xdt == MBT_E4M3) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 h = Elem<MBT_F16>::widen2(
                    e4m3x2_to_half2((i < 2 ? raw[t].x : raw[t].y) >> (16 * (i & 1))));
                f[2 * i] = h.x;
                f[2 * i + 1] = h.y;
            }
            if (in) factor = __ldg(a.xs + (t0 + t) * a.x_groups + (a.x_row_scale ? 0 : k / 128));
        } else if (a.xdt == MBT_BF16) {
            unpack<MBT_BF16>(raw[t], f);
        } else {
            unpack<MBT_F16>(raw[t], f);
        }
        uint32_t amax = 0;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            amax = max(amax, magnitude(f[i]));
            sum += f[i];
        }
#pragma unroll
        for (int o = 1; o < G / 8; o <<= 1) {
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        }
        // 2^e brings the group's largest value into [2^14, 2^15); a group of
        // zeros or with an infinity or NaN is left as it is
        const int eb = static_cast<int>(amax >> 23);
        const int e = amax == 0 || eb == 255 ? 0 : min(max(14 - (eb - 127), -126), 126);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= up;
        const uint4 v = make_uint4(Elem<MBT_F16>::round2(f[0], f[4]),
                                   Elem<MBT_F16>::round2(f[1] * 0.0625f, f[5] * 0.0625f),
                                   Elem<MBT_F16>::round2(f[2], f[6]),
                                   Elem<MBT_F16>::round2(f[3] * 0.0625f, f[7] * 0.0625f));
        const uint32_t dst = xbuf + 16u * static_cast<uint32_t>(((u >> 2) * tokens + t) * 4 + (u & 3));
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y),
                     "r"(v.z), "r"(v.w)
                     : "memory");
        if (u % (G / 8) == 0) {
            const uint32_t m = meta + 64u * static_cast<uint32_t>(u / (G / 8)) + 8u * t;
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(m), "f"(down * factor),
                         "f"(sum * factor * 5.9604644775390625e-8f)
                         : "memory");
        }
    }
}

// acc += s 2^24 (p 2^-e - z 2^-24 sum x) of the lane's two rows of q and of x; p = 0.
__device__ __forceinline__ void flush_group(float (&acc)[4], float (&p)[4], uint32_t scales,
                                            uint32_t meta) {
    const uint4 m = lds128(meta), v = lds128(scales);
    const float f0 = __uint_as_float(m.x), x0 = __uint_as_float(m.y);
    const float f1 = __uint_as_float(m.z), x1 = __uint_as_float(m.w);
    const float sl = __uint_as_float(v.x), zl = __uint_as_float(v.y);
    const float sh = __uint_as_float(v.z), zh = __uint_as_float(v.w);
    acc[0] += sl * (p[0] * f0 - zl * x0);
    acc[1] += sl * (p[1] * f1 - zl * x1);
    acc[2] += sh * (p[2] * f0 - zh * x0);
    acc[3] += sh * (p[3] * f1 - zh * x1);
    p[0] = p[1] = p[2] = p[3] = 0.f;
}

template <int G, bool S32>
__global__ void __launch_bounds__(kW4Threads, 2)
    mbt_w4_kernel(const __grid_constant__ CUtensorMap map, const W4Args a) {
    constexpr int kStages = W4Seg<G>::kStages;
    extern __shared__ __align__(1024) unsigned char dyn_smem[];
    __shared__ __align__(8) uint64_t bars[2 * kStages + 2 * kW4Segs];
    __shared__ int abort_flag;
    __shared__ float red[kW4Tokens][kW4Rows];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kW4Tokens;
    const int tokens = static_cast<int>(a.T - t0 < kW4Tokens ? a.T - t0 : kW4Tokens);
    const int rank = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.slices));
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(a.slices)) * kW4Rows;
    const int64_t segs = (a.K + kW4Seg - 1) / kW4Seg;
    const int64_t seg0 = rank * segs / a.slices, seg1 = (rank + 1) * segs / a.slices;
    const int64_t all_steps = (a.K + kW4Step - 1) / kW4Step;
    const int64_t step0 = seg0 * 2, step1 = seg1 * 2 < all_steps ? seg1 * 2 : all_steps;
    W4Rings r;
    r.q = (smem_u32(dyn_smem) + (kSwizzleAtomBytes - 1)) & ~uint32_t(kSwizzleAtomBytes - 1);
    r.x = r.q + kStages * kW4StageBytes;
    r.x_bytes = static_cast<uint32_t>(kW4Seg * 2 * tokens);
    r.seg_bytes = r.x_bytes + W4Seg<G>::kMeta + W4Seg<G>::kScales;
    r.full_q = smem_u32(bars);
    r.empty_q = r.full_q + 8 * kStages;
    r.full_x = r.empty_q + 8 * kStages;
    r.empty_x = r.full_x + 8 * kW4Segs;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(r.full_q + 8 * i, 1);
            mbar_init(r.empty_q + 8 * i, kW4Consumers);
        }
        for (int i = 0; i < kW4Segs; ++i) {
            mbar_init(r.full_x + 8 * i, 64);
            mbar_init(r.empty_x + 8 * i, kW4Consumers);
        }
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const WaitCtl w{kDefaultWaitBudgetNs, &abort_flag, a.status};

    if (warp == kW4Consumers) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 1;
            int64_t issued = 0;
            for (int64_t s = step0; s < step1; ++s) {
                if (!wait_bounded(r.empty_q + 8 * stage, phase, w, true)) {
                    report_timeout(w, 0, stage, phase);
                    abort_flag = 1;
                    // the copies still in flight land before the CTA leaves
                    for (int64_t k = issued > kStages ? issued - kStages : 0; k < issued; ++k)
                        wait_bounded(r.full_q + 8 * static_cast<uint32_t>(k % kStages),
                                     static_cast<uint32_t>(k / kStages & 1), w, false);
                    break;
                }
                mbar_arrive_expect_tx(r.full_q + 8 * stage, kW4StageBytes);
                tma_load_2d(r.q + stage * kW4StageBytes, &map, static_cast<int32_t>(s * (kW4Step / 2)),
                            static_cast<int32_t>(row0), r.full_q + 8 * stage);
                ++issued;
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
        }
    } else if (warp > kW4Consumers) {
        const int u = static_cast<int>(threadIdx.x) - 32 * (kW4Consumers + 1);
        uint32_t buf = 0, phase = 1;
        for (int64_t s = seg0; s < seg1; ++s) {
            // (a warp goes on, or gives up, as one)
            if (!__all_sync(0xffffffffu, wait_bounded(r.empty_x + 8 * buf, phase, w, true))) {
                report_timeout(w, 0, kMaxStages + buf, phase);
                abort_flag = 1;
                break;
            }
            const uint32_t at = r.x + buf * r.seg_bytes;
            stage_scales<G, S32>(a, s, row0, u, at + r.x_bytes + W4Seg<G>::kMeta);
            stage_x<G>(a, s, t0, tokens, u, at, at + r.x_bytes);
            mbar_arrive(r.full_x + 8 * buf);
            if (++buf == kW4Segs) buf = 0, phase ^= 1;
        }
    } else {
        // ldmatrix: lane l gives the address of row l % 8 (+ 8 for odd eights) of chunk l / 16
        const int lrow = warp * 16 + (lane & 15);
        const uint32_t laddr = static_cast<uint32_t>(lrow) * 128u;
        const uint32_t lchunk = static_cast<uint32_t>(lane >> 4), lswz = static_cast<uint32_t>(lrow & 7);
        const int tok = lane >> 2 < tokens ? lane >> 2 : tokens - 1;
        const uint32_t xlane = static_cast<uint32_t>(tok * 4 + (lane & 3)) * 16u;
        const uint32_t xchunk = static_cast<uint32_t>(tokens) * 64u;
        constexpr int kN = kW4Step / G;
        float acc[4] = {0.f, 0.f, 0.f, 0.f}, p[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t stage = 0, phase = 0, buf = 0, xphase = 0;
        for (int64_t s = step0; s < step1; ++s) {
            bool ok = (s & 1) || wait_bounded(r.full_x + 8 * buf, xphase, w, true);
            ok = ok && wait_bounded(r.full_q + 8 * stage, phase, w, true);
            if (!__all_sync(0xffffffffu, ok)) {
                report_timeout(w, 1, stage, phase);
                abort_flag = 1;
                break;
            }
            const uint32_t q = r.q + stage * kW4StageBytes + laddr;
            const uint32_t half = static_cast<uint32_t>(s & 1);
            const uint32_t seg = r.x + buf * r.seg_bytes;
            const uint32_t x = seg + half * 8u * xchunk + xlane;
            const uint32_t meta = seg + r.x_bytes + half * kN * 64u + (lane & 3) * 16u;
            const uint32_t scales = seg + r.x_bytes + W4Seg<G>::kMeta +
                                    half * kN * (8u * kW4Rows) + static_cast<uint32_t>(warp * 128 + (lane >> 2) * 16);
            uint32_t v[4][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) ldmatrix_x4(v[c], q + ((2u * c + lchunk) ^ lswz) * 16u);
            __syncwarp();
            if (lane == 0) mbar_arrive(r.empty_q + 8 * stage);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const uint32_t wl = v[c >> 1][2 * (c & 1)], wh = v[c >> 1][2 * (c & 1) + 1];
                const uint4 b = lds128(x + static_cast<uint32_t>(c) * xchunk);
                const uint32_t wl8 = wl >> 8, wh8 = wh >> 8;
                mma_f16(p, wl & 0x000f000fu, wh & 0x000f000fu, wl & 0x00f000f0u, wh & 0x00f000f0u, b.x, b.y);
                mma_f16(p, wl8 & 0x000f000fu, wh8 & 0x000f000fu, wl8 & 0x00f000f0u, wh8 & 0x00f000f0u, b.z, b.w);
                if ((c + 1) * 32 % G == 0)
                    flush_group(acc, p, scales + c * 32 / G * (8u * kW4Rows), meta + c * 32 / G * 64u);
            }
            if (++stage == kStages) stage = 0, phase ^= 1;
            if ((s & 1) || s + 1 == step1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(r.empty_x + 8 * buf);
                if (++buf == kW4Segs) buf = 0, xphase ^= 1;
            }
        }
        const int n = warp * 16 + (lane >> 2), t = 2 * (lane & 3);
        red[t][n] = acc[0];
        red[t + 1][n] = acc[1];
        red[t][n + 8] = acc[2];
        red[t + 1][n + 8] = acc[3];
    }
    // the slices' sums, in rank order; CTA `rank` finishes its share of the rows
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    __syncwarp();
    cluster.sync();
    const int rows = kW4Rows / a.slices;
    for (int i = threadIdx.x; i < tokens * rows; i += kW4Threads) {
        const int t = i / rows, n = rank * rows + i % rows;
        if (row0 + n >= a.N) continue;
        float y = 0.f;
        for (int c = 0; c < a.slices; ++c) y += *cluster.map_shared_rank(&red[t][n], c);
        store_any(a.out, a.odt, (t0 + t) * a.ld_out + row0 + n, y);
    }
    cluster.sync();   // no CTA leaves while its sums may still be read
}

bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

uintptr_t type_bytes(int dtype) { return dtype == MBT_F32 ? 4 : dtype == MBT_E4M3 ? 1 : 2; }

__global__ void mbt_w4_zero_kernel(void *out, int dtype, int64_t N, int64_t ld) {
    for (int64_t n = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; n < N;
         n += static_cast<int64_t>(gridDim.x) * blockDim.x)
        store_any(out, dtype, blockIdx.y * ld + n, 0.f);
}

template <int G, bool S32>
cudaError_t launch_w4(const CUtensorMap &map, const W4Args &a, dim3 grid, cudaStream_t stream) {
    const int tokens = static_cast<int>(std::min<int64_t>(a.T, kW4Tokens));
    constexpr int kFixed = kSwizzleAtomBytes + W4Seg<G>::kStages * kW4StageBytes +
                           kW4Segs * (W4Seg<G>::kMeta + W4Seg<G>::kScales);
    const size_t smem = kFixed + kW4Segs * kW4Seg * 2 * tokens;
    static_assert(kFixed + kW4Segs * kW4Seg * 2 * kW4Tokens <= kW4MaxSmem,
                  "the largest launch fits the limit set below");
    static std::atomic<bool> raised[64];   // per device: the kernel's shared-memory limit is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !raised[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(mbt_w4_kernel<G, S32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kW4MaxSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) raised[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kW4Threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(a.slices);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, mbt_w4_kernel<G, S32>, map, a);
}

template <int G>
cudaError_t launch_w4_group(const CUtensorMap &map, const W4Args &a, dim3 grid, cudaStream_t stream) {
    return a.sdt == MBT_F32 ? launch_w4<G, true>(map, a, grid, stream)
                            : launch_w4<G, false>(map, a, grid, stream);
}

}  // namespace
}  // namespace mbt

extern "C" int tile_w4_matvec(const void *x, const float *x_scales, const uint8_t *q,
                              const void *scales, const uint8_t *zeros, void *out, int64_t T,
                              int64_t N, int64_t K, int64_t ld_x, int64_t ld_q, int64_t ld_out,
                              int group, int x_group, int dtype, int scale_dtype, int out_dtype,
                              void *stream) {
    using namespace mbt;
    if (T < 0 || N < 0 || K < 0 || T > 0x7fffffff || N > 0x7fffffff || K > 0x7fffffff)
        return MBT_ERR_ARG;
    if (dtype != MBT_F16 && dtype != MBT_BF16 && dtype != MBT_E4M3) return MBT_ERR_ARG;
    if (scale_dtype < MBT_F16 || scale_dtype > MBT_F32 || out_dtype < MBT_F16 || out_dtype > MBT_F32)
        return MBT_ERR_ARG;
    if (K % 32 != 0 || (group != 32 && group != 64 && group != 128)) return MBT_ERR_UNSUPPORTED;
    if (ld_x == 0) ld_x = K;
    if (ld_q == 0) ld_q = K / 2;
    if (ld_out == 0) ld_out = N;
    if (ld_x < K || ld_q < K / 2 || ld_out < N || ld_x > (1ll << 40) || ld_q >= (1ll << 40) ||
        ld_out > (1ll << 40))
        return MBT_ERR_ARG;
    if (dtype == MBT_E4M3) {
        if (x_group != 0 && x_group != 128) return MBT_ERR_UNSUPPORTED;
    } else if (x_scales || x_group != 0) {
        return MBT_ERR_ARG;
    }
    if (T == 0 || N == 0) return MBT_OK;
    if (!out || (K > 0 && (!x || !q || !scales || (dtype == MBT_E4M3 && !x_scales))))
        return MBT_ERR_ARG;
    if (!aligned(x, type_bytes(dtype)) || !aligned(scales, type_bytes(scale_dtype)) ||
        !aligned(out, type_bytes(out_dtype)) || !aligned(x_scales, 4) || !aligned(q, 16) ||
        ld_q % 16 != 0)
        return MBT_ERR_ALIGN;
    const int64_t token_blocks = (T + kW4Tokens - 1) / kW4Tokens;
    if (token_blocks > 65535 || (K == 0 && T > 65535)) return MBT_ERR_UNSUPPORTED;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (K == 0) {
        const dim3 grid(static_cast<unsigned>(std::min<int64_t>((N + 255) / 256, 1024)),
                        static_cast<unsigned>(T));
        mbt_w4_zero_kernel<<<grid, 256, 0, st>>>(out, out_dtype, N, ld_out);
        return cudaGetLastError() == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
    }
    int sms = 0, optin = 0;
    int rc = device_limits(&sms, &optin);
    if (rc != MBT_OK) return rc;
    W4Args a{};
    rc = device_status_word(&a.status);
    if (rc != MBT_OK) return rc;
    a.x = x;
    a.s = scales;
    a.z = zeros;
    a.xs = x_scales;
    a.out = out;
    a.T = T;
    a.N = N;
    a.K = K;
    a.ld_x = ld_x;
    a.ld_out = ld_out;
    a.groups = (K + group - 1) / group;
    a.x_groups = x_group ? (K + x_group - 1) / x_group : 1;
    a.xdt = dtype;
    a.sdt = scale_dtype;
    a.odt = out_dtype;
    a.x_row_scale = x_group == 0;
    // a segment's scales of a row as vectors: whole ones, aligned in every row
    const int per_seg = kW4Seg / group;
    const int vec = std::min<int>(per_seg, 16 / static_cast<int>(type_bytes(scale_dtype)));
    a.vec_scales = a.groups % vec == 0 && aligned(scales, vec * type_bytes(scale_dtype));
    a.vec_zeros = a.groups % 4 == 0 && aligned(zeros, 4);
    const uintptr_t xb = type_bytes(dtype);
    a.vec_x = aligned(x, 8 * xb) && (T == 1 || ld_x * static_cast<int64_t>(xb) % (8 * static_cast<int64_t>(xb)) == 0);
    // Slices along K until there are CTAs for 1.6 per SM (two fit, and loads in
    // flight on every SM are what counts), each at least one segment of x.
    const int64_t blocks = (N + kW4Rows - 1) / kW4Rows * token_blocks;
    const int64_t segs = (K + kW4Seg - 1) / kW4Seg;
    int slices = 1;
    while (slices < kW4MaxSlices && slices * 2 <= segs && blocks * slices * 10 < 16 * sms) slices *= 2;
    a.slices = slices;
    if ((N + kW4Rows - 1) / kW4Rows * slices > 0x7fffffff) return MBT_ERR_UNSUPPORTED;
    alignas(64) CUtensorMap map;
    rc = encode_bytes_map(&map, q, N, K / 2, ld_q, kW4Rows);
    if (rc != MBT_OK) return rc;
    const dim3 grid(static_cast<unsigned>((N + kW4Rows - 1) / kW4Rows * slices),
                    static_cast<unsigned>(token_blocks));
    const cudaError_t e = group == 32   ? launch_w4_group<32>(map, a, grid, st)
                          : group == 64 ? launch_w4_group<64>(map, a, grid, st)
                                        : launch_w4_group<128>(map, a, grid, st);
    return e == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
}
