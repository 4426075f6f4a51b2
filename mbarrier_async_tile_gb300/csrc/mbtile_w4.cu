// tile_w4_matvec: products of a few rows of activations with a matrix held in
// 4 bits, y[t, n] = sum_k x[t, k] (q[n, k] - z[n, k / g]) s[n, k / g].
//
// The matrix is read once and each of its elements used at most eight times:
// device memory bounds the large products, latency the small ones.  One to four
// rows of x and few elements have a kernel of their own, mbtile_w4_few.cuh.  Here
// fp16 16384 x 16384 by groups of 64 with zero points and 8 rows of x takes 42.1 us,
// 3.5 TB/s, and e4m3 8191 x 8192 by groups of 32 and 3 rows 17.0 us, 2.2 TB/s (replayed
// from graphs, q from device memory): the ring
// alone streams the former in 25 us, the consumers' conversions and scales take
// 53 % of the issue slots beside it, and the kernels before and after it and the
// start some 7 us.
//
// The work is cut into units of 64 rows of q by a slice of K short enough for
// its part of x to stay in shared memory; slice by slice, the units are dealt out
// evenly to the CTAs (two per SM), so that a CTA takes its part of x once or twice.
// A small kernel before this one brings x into the form that the tensor
// instructions read (done by the CTAs themselves it took 5 of 40 us at 16384 x
// 16384 and 8 rows of x); this one starts while that runs and loads its first
// stages of q meanwhile.  Warp roles:
//   8 consumer warps: 16 rows each, the two halves of a step's columns;
//   a producer thread: steps of 64 rows x 512 columns (two boxes of 64 x 128
//   bytes) of q by bulk tensor copies into a ring of 128-byte-swizzled stages, and
//   a slice's part of x by one bulk copy;
//   2 staging warps: a step's scales and zero points, converted once per CTA
//   into the same stages, from registers loaded several steps ahead;
//   a flush warp: takes a finished unit's sums from the consumers and, where K is
//   sliced, writes them to the workspace, whose slices a second, small kernel adds
//   up in order.  (With tickets the last slice's CTA did that: its one warp took 8
//   us for 11 slices and 8 rows of x.)
//
// The products are m16n8k16 tensor instructions with 16 rows of q as A and up to
// eight rows of x as B.  (Tcgen05's smallest tile has 64 rows against 8 columns
// and takes its operands from shared memory or its own memory, where q would first
// have to be written back in 16 bits; here q goes from registers.  The e4m3 form
// of the instruction, for which a nibble is a code as it stands, is carried out as
// two fp16 ones with conversions here: measured, 1.4 times the instructions.)
//
// An A element is q - z as fp16, exactly, by the known addition to a power of two whose
// last place is one (for 4-bit weights in fp16: Kim, Henry, Fahim, Awadalla, "Who Says
// Elephants Can't Run", SustaiNLP 2022): a 4-bit value put into the mantissa of
// 1024 (bits 0..3) is 1024 + q, from which 1024 + z is subtracted; in bits 4..7
// it is 1024 + 16 q, which a multiplication by 1/16 and a subtraction of 64 + z
// take to the same.  Eight values cost four ANDs with ORs, a shift and four
// packed fp16 operations.  (Left as fp16 subnormals the values would need no
// arithmetic, but the tensor unit then aligns its products by the subnormals'
// nominal exponent and loses up to ten bits: measured, errors of 80 u times the
// sum of magnitudes in rows with outliers, against 0.3 u.)  Which k goes where in
// the instruction is free as long as A and B agree: a 16-byte chunk of a row (32
// columns) is read by ldmatrix as if it held 16-bit elements, which gives the
// lane of column pair j the bytes 4j..4j+3, columns 8j..8j+7; nibbles i and
// i + 4 share a half pair.
//
// x is scaled by a power of two per row and group (16-bit inputs of any range
// then fit fp16: values below 2^-29 of the group's largest lose bits, less than
// fp32 sums do), and each group's product p is taken back in fp32:
//   acc += s 2^-e p.
#include <algorithm>
#include <atomic>

#include "mbtile_elem.cuh"
#include "mbtile_layer.h"
#include "mbtile_ptx.cuh"

namespace mbt {
namespace {

constexpr int kW4Rows = 64;               // rows of q per unit
constexpr int kW4Step = 512;              // columns per stage
constexpr int kW4Consumers = 8;           // warps
constexpr int kW4Stagers = 64;            // threads, one per row of q
constexpr int kW4Threads = 32 * (kW4Consumers + 2) + kW4Stagers;
constexpr int kW4BoxBytes = kW4Rows * kBoxRowBytes;
constexpr int kW4QBytes = 2 * kW4BoxBytes;
constexpr int kW4Tokens = 8;
// Bytes of a unit's part of x, which with the stages leave room for two CTAs per SM.
constexpr int kW4XBytes = 36352;
constexpr int64_t kW4MostScratch = 128 << 20;   // bytes of workspace, unless eight rows of x take more

struct W4Args {
    const uint8_t *q;           // few rows of x: q read without a tensor map
    int64_t ld_q;
    int32_t group_shift;        // log2 of the columns a scale covers
    int32_t few_split;          // warps of a CTA that share a row of q
    const void *x;
    const void *s;
    const uint8_t *z;
    const float *xs;
    unsigned char *xb;          // x as B elements, see x_block
    void *out;
    int64_t T, N, K, ld_x, ld_out;
    int64_t groups, x_groups;   // scales of a row of q, of a row of x
    int32_t xdt, sdt, odt;
    int32_t x_row_scale;        // e4m3: a scale per row of x, else per 128 columns
    int32_t slices;             // of K, in whole steps
    int32_t slice_steps;        // steps of the longest slice
    int32_t x_rows;             // most rows of x in a unit
    int32_t blocks;             // of 64 rows of q
    int32_t units;              // eights of rows of x * slices * blocks
    int32_t steps;              // of K
    float *partial;             // [t][slice][64 blocks], with more than one slice
    int32_t vec_scales;         // a step's 16-bit scales of a row are aligned vectors
    int32_t vec_zeros;
    int32_t vec_x;              // eight columns of x are one aligned vector
    int32_t *status;
};

}  // namespace
}  // namespace mbt

#include "mbtile_w4_few.cuh"

namespace mbt {
namespace {

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// c = a b + (FIRST ? 0 : c)
template <bool FIRST>
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    const float z = 0.f;
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(FIRST ? z : c[0]),
          "f"(FIRST ? z : c[1]), "f"(FIRST ? z : c[2]), "f"(FIRST ? z : c[3]));
}

template <int G>
struct W4Step {
    static constexpr int kGroups = kW4Step / G;
    static constexpr int kScales = kGroups * kW4Rows * 8;   // {s, fp16 pair 1024 + z} per group and row
    static constexpr int kStage = kW4QBytes + kScales;      // a multiple of 1024
    static constexpr int kStages = G == 128 ? 4 : 3;
};

// Code that runs once per CTA, or for unaligned arrays only, is kept out of line
// or in rolled loops: the first pass over any instruction misses the caches.

// Eight columns of x at any alignment.
__device__ __noinline__ uint4 load_x_elements(const void *x, int xdt, int64_t at) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (xdt == MBT_E4M3) {
        const uint8_t *p = static_cast<const uint8_t *>(x) + at;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            v.x |= static_cast<uint32_t>(p[i]) << (8 * i);
            v.y |= static_cast<uint32_t>(p[4 + i]) << (8 * i);
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(x) + at;
        v.x = p[0] | static_cast<uint32_t>(p[1]) << 16;
        v.y = p[2] | static_cast<uint32_t>(p[3]) << 16;
        v.z = p[4] | static_cast<uint32_t>(p[5]) << 16;
        v.w = p[6] | static_cast<uint32_t>(p[7]) << 16;
    }
    return v;
}

__device__ __forceinline__ uint4 load_x(const W4Args &a, int64_t at) {
    if (!a.vec_x) return load_x_elements(a.x, a.xdt, at);
    if (a.xdt == MBT_E4M3) {
        const uint2 q = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(a.x) + at));
        return make_uint4(q.x, q.y, 0, 0);
    }
    return __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + at));
}

// Eight columns of x (as loaded) as B elements, scaled by 2^e with the e of their
// group, `lanes` neighbouring lanes, which is returned as 2^-e in *down.
__device__ __forceinline__ uint4 convert_x(uint4 v, int xdt, int lanes, float *down) {
    float f[8];
    if (xdt == MBT_E4M3) {
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) h[j] = e4m3x2_to_half2((j < 2 ? v.x : v.y) >> (16 * (j & 1)));
        v = make_uint4(h[0], h[1], h[2], h[3]);
    }
    // 16-bit magnitudes order as integers, NaN above infinity
    uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                          __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    m = max(m & 0xffffu, m >> 16);
#pragma unroll
    for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    uint32_t top;                           // bits of the largest magnitude, as fp32
    if (xdt == MBT_BF16) {
        unpack<MBT_BF16>(v, f);
        top = m << 16;
    } else {
        unpack<MBT_F16>(v, f);
        top = __float_as_uint(Elem<MBT_F16>::widen2(m).x);
    }
    // 2^e brings the group's largest value into [2^14, 2^15); a group of zeros or
    // with an infinity or NaN is left as it is
    const int eb = static_cast<int>(top >> 23);
    const int e = top == 0 || eb == 255 ? 0 : min(14 - (eb - 127), 126);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= up;
    *down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    return make_uint4(Elem<MBT_F16>::round2(f[0], f[4]), Elem<MBT_F16>::round2(f[1], f[5]),
                      Elem<MBT_F16>::round2(f[2], f[6]), Elem<MBT_F16>::round2(f[3], f[7]));
}

// x as B elements, step by step: a block for every eight rows of x and 512 columns,
// the rows kXPitch bytes apart (64 bytes apart in the banks: a warp's reads of 8
// rows x 64 bytes do not collide), then 2^-e of each group, [group][8].
constexpr int kXPitch = kW4Step * 2 + 64;
__host__ __device__ constexpr int x_block(int rows, int group) {
    return rows * kXPitch + kW4Step / group * kW4Tokens * 4;
}

constexpr int kW4XThreads = 128;

// Eight columns of one row of x per thread; a CTA holds whole steps' halves of a row.
template <int G>
__global__ void __launch_bounds__(kW4XThreads) mbt_w4_x_kernel(const __grid_constant__ W4Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // what ran before is done: the main kernel may start, and read q and the scales
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int u = static_cast<int>(blockIdx.x) * kW4XThreads + static_cast<int>(threadIdx.x);
    const int t = static_cast<int>(blockIdx.y);
    const int64_t k = 8ll * u;
    if (k >= static_cast<int64_t>(a.steps) * kW4Step) return;   // whole warps
    uint4 raw = make_uint4(0, 0, 0, 0);
    float xs = 1.f, down;
    if (k < a.K) {
        raw = load_x(a, t * a.ld_x + k);
        if (a.xs) xs = __ldg(a.xs + t * a.x_groups + (a.x_row_scale ? 0 : k / 128));
    }
    const uint4 v = convert_x(raw, a.xdt, G / 8, &down);
    const int64_t eight = t / kW4Tokens, step = u / (kW4Step / 8);
    const int row = t % kW4Tokens, rows = min(static_cast<int>(a.T - eight * kW4Tokens), kW4Tokens);
    const int c = u % (kW4Step / 8);
    // (every eight but the last has eight rows)
    unsigned char *block = a.xb + (eight * a.steps * x_block(kW4Tokens, G)) + step * x_block(rows, G);
    *reinterpret_cast<uint4 *>(block + row * kXPitch + c * 16) = v;
    if (c % (G / 8) == 0)
        reinterpret_cast<float *>(block + rows * kXPitch)[c / (G / 8) * kW4Tokens + row] = down * xs;
}

// Element i of a row's scales or zero points, any type.
__device__ __noinline__ uint32_t load_scale_bits(const void *s, int sdt, int64_t at) {
    return sdt == MBT_F32 ? __ldg(static_cast<const uint32_t *>(s) + at)
                          : __ldg(static_cast<const uint16_t *>(s) + at);
}

// A staging thread's row of a step's scales and zero points, as loaded.
template <int G>
struct RowScales {
    static constexpr int kGroups = kW4Step / G;
    uint32_t s[kGroups / 2];                // 16-bit scales
    uint32_t z[kGroups / 4];

    __device__ __forceinline__ void load(const W4Args &a, int64_t row, int64_t g0) {
#pragma unroll
        for (int i = 0; i < kGroups / 2; ++i) s[i] = 0;
#pragma unroll
        for (int i = 0; i < kGroups / 4; ++i) z[i] = 0x08080808u;
        if (row >= a.N) return;
        const int64_t at = row * a.groups + g0;
        const bool whole = g0 + kGroups <= a.groups;
        if (a.vec_scales && whole) {
            const uint16_t *p = static_cast<const uint16_t *>(a.s) + at;
            if constexpr (kGroups == 4) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
                s[0] = v.x, s[1] = v.y;
            } else {
#pragma unroll
                for (int i = 0; i < kGroups / 8; ++i) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
                    s[4 * i] = v.x, s[4 * i + 1] = v.y, s[4 * i + 2] = v.z, s[4 * i + 3] = v.w;
                }
            }
        }
        if (a.z && a.vec_zeros && whole) {
#pragma unroll
            for (int i = 0; i < kGroups / 4; ++i)
                z[i] = __ldg(reinterpret_cast<const uint32_t *>(a.z + at) + i);
        }
    }

    // Rows n and n + 8 of a warp's 16 lie side by side, so that one 16-byte read
    // gives a consumer lane both of its rows.
    __device__ __forceinline__ void store(const W4Args &a, int64_t row, int64_t g0, int local,
                                          uint2 *dst) const {
        const int slot = (local & ~15) | (local & 7) << 1 | (local >> 3 & 1);
        const bool whole = g0 + kGroups <= a.groups;
        if (a.vec_scales && whole && (a.z == nullptr || a.vec_zeros)) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const uint32_t b = s[i / 2] >> (16 * (i & 1));
                const float v = a.sdt == MBT_BF16 ? __uint_as_float(b << 16) : Elem<MBT_F16>::widen2(b).x;
                const uint32_t zero = (0x6400u | (z[i / 4] >> (8 * (i % 4)) & 15u)) * 0x10001u;
                dst[i * kW4Rows + slot] = make_uint2(__float_as_uint(v), zero);
            }
            return;
        }
        // other types and alignments, and a row's end (0 past it): element by element
#pragma unroll 1
        for (int i = 0; i < kGroups; ++i) {
            const bool in = row < a.N && g0 + i < a.groups;
            const int64_t at = row * a.groups + g0 + i;
            const uint32_t b = in ? load_scale_bits(a.s, a.sdt, at) : 0u;
            const uint32_t zero = in && a.z ? a.z[at] & 15u : 8u;
            const float v = a.sdt == MBT_F32    ? __uint_as_float(b)
                            : a.sdt == MBT_BF16 ? __uint_as_float(b << 16)
                                                : Elem<MBT_F16>::widen2(b).x;
            dst[i * kW4Rows + slot] = make_uint2(__float_as_uint(v), (0x6400u | zero) * 0x10001u);
        }
    }
};

__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2 *>(&v); }
__device__ __forceinline__ uint32_t as_bits(__half2 v) { return *reinterpret_cast<const uint32_t *>(&v); }

// The conversion's constants, in registers: an instruction takes one immediate,
// and the compiler, which knows the values, would move the others in every time.
struct Nibbles {
    uint32_t low, high, k1024, sixteenth;
    __device__ __forceinline__ Nibbles() {
        asm volatile("mov.b32 %0, 0x000f000f;" : "=r"(low));
        asm volatile("mov.b32 %0, 0x00f000f0;" : "=r"(high));
        asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k1024));
        asm volatile("mov.b32 %0, 0x2c002c00;" : "=r"(sixteenth));
    }
    static __device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
        uint32_t r;
        asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
        return r;
    }
    // nibbles 0 and 4 of w, less z (z1024 = 1024 + z), from bits 0..3 of each half
    __device__ __forceinline__ uint32_t lower(uint32_t w, __half2 z1024) const {
        return as_bits(__hsub2(as_half2(and_or(w, low, k1024)), z1024));
    }
    // nibbles 1 and 5 of w, less z (z64 = -(64 + z)), from bits 4..7 of each half
    __device__ __forceinline__ uint32_t upper(uint32_t w, __half2 z64) const {
        return as_bits(__hfma2(as_half2(and_or(w, high, k1024)), as_half2(sixteenth), z64));
    }
};

// wait_bounded with its first probe in line.
__device__ __forceinline__ bool arrived(uint32_t bar, uint32_t parity, const WaitCtl &w) {
    return mbar_try_wait(bar, parity) || wait_bounded(bar, parity, w, true);
}

// Four consecutive outputs of row t, those below N.
__device__ __noinline__ void store_y(const W4Args &a, int64_t t, int64_t n, float4 y) {
#pragma unroll 1
    for (int k = 0; k < 4 && n + k < a.N; ++k) {
        store_any(a.out, a.odt, t * a.ld_out + n + k, y.x);
        y.x = y.y, y.y = y.z, y.z = y.w;
    }
}

// What unit i is.  (All counts fit 32 bits, and a 64-bit division is a hundred
// instructions.)
struct W4Unit {
    int t0, block, slice, step0, step1;   // first row of x, block of q, slice, its steps
    int tokens;
    __device__ __forceinline__ W4Unit(const W4Args &a, int i) {
        const int r = i / a.blocks;
        block = i - r * a.blocks;
        const int eight = r / a.slices;
        slice = r - eight * a.slices;
        t0 = eight * kW4Tokens;
        tokens = min(static_cast<int>(a.T) - t0, kW4Tokens);
        // the first `longer` slices have a step more than the others
        const int each = a.steps / a.slices, longer = a.steps - each * a.slices;
        step0 = slice * each + min(slice, longer);
        step1 = step0 + each + (slice < longer);
    }
};

template <int G>
__global__ void __launch_bounds__(kW4Threads, 2)
    mbt_w4_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ W4Args a) {
    extern __shared__ __align__(1024) unsigned char dyn_smem[];
    constexpr int kStages = W4Step<G>::kStages;
    __shared__ __align__(8) uint64_t bars[2 * kStages + 4];
    __shared__ int abort_flag;
    __shared__ __align__(16) float red[2][kW4Tokens][kW4Rows];   // [half of the columns]
    using Step = W4Step<G>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // (aligned by its address in the shared window, as the swizzle is)
    unsigned char *const ring = dyn_smem + ((0u - smem_u32(dyn_smem)) & (kSwizzleAtomBytes - 1));
    unsigned char *const xbuf = ring + Step::kStages * Step::kStage;
    const uint32_t full = smem_u32(bars), empty = full + 8 * kStages;
    const uint32_t full_r = empty + 8 * kStages, empty_r = full_r + 8;
    const uint32_t full_x = empty_r + 8, empty_x = full_x + 8;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(full + 8 * i, 1 + kW4Stagers);
            mbar_init(empty + 8 * i, kW4Consumers);
        }
        mbar_init(full_r, kW4Consumers);
        mbar_init(empty_r, 1);
        mbar_init(full_x, 1);
        mbar_init(empty_x, kW4Consumers);
        abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();
    // The kernel before (mbt_w4_x_kernel) has waited for everything before it, so q,
    // the scales and the zero points may be read; x as B elements and the
    // workspace's sums only after griddepcontrol.wait.  The slices' sums' kernel
    // may be set up from now on.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const WaitCtl w{kDefaultWaitBudgetNs, &abort_flag, a.status};
    const int u0 = static_cast<int>(static_cast<uint64_t>(blockIdx.x) * a.units / gridDim.x);
    const int u1 = static_cast<int>(static_cast<uint64_t>(blockIdx.x + 1) * a.units / gridDim.x);

    if (warp == kW4Consumers) {                 // producer
        if (lane != 0) return;
        uint32_t stage = 0, phase = 1, xphase = 1;
        int64_t issued = 0;
        int staged = -1, x_copies = 0;
        auto give_up = [&](uint32_t st, uint32_t ph) {
            report_timeout(w, 0, st, ph);
            abort_flag = 1;
            // the copies still in flight land before the CTA leaves (the stagers'
            // arrivals may be missing: the wait is bounded)
            for (int64_t k = issued > kStages ? issued - kStages : 0; k < issued; ++k)
                wait_bounded(full + 8 * static_cast<uint32_t>(k % kStages),
                             static_cast<uint32_t>(k / kStages & 1), w, false);
            if (x_copies) wait_bounded(full_x, static_cast<uint32_t>(x_copies - 1) & 1u, w, false);
        };
        for (int i = u0; i < u1; ++i) {
            const W4Unit u(a, i);
            for (int s = u.step0; s < u.step1; ++s) {
                if (!arrived(empty + 8 * stage, phase, w)) return give_up(stage, phase);
                mbar_arrive_expect_tx(full + 8 * stage, kW4QBytes);
                const uint32_t dst = smem_u32(ring) + stage * Step::kStage;
                const int32_t col = static_cast<int32_t>(s * (kW4Step / 2));
                const int32_t row = static_cast<int32_t>(u.block * kW4Rows);
                tma_load_2d(dst, &map, col, row, full + 8 * stage);
                tma_load_2d(dst + kW4BoxBytes, &map, col + kBoxRowBytes, row, full + 8 * stage);
                ++issued;
                if (++stage == kStages) stage = 0, phase ^= 1;
                // a new slice's x, behind as much of q as the ring takes at first
                if (i / a.blocks != staged && (s + 1 == u.step1 || s + 1 - u.step0 == kStages)) {
                    staged = i / a.blocks;
                    asm volatile("griddepcontrol.wait;" ::: "memory");
                    if (!arrived(empty_x, xphase, w)) return give_up(kStages, xphase);
                    xphase ^= 1;
                    const int block = x_block(u.tokens, G);
                    const uint32_t bytes = static_cast<uint32_t>((u.step1 - u.step0) * block);
                    mbar_arrive_expect_tx(full_x, bytes);
                    bulk_load_1d(smem_u32(xbuf),
                                 a.xb + static_cast<int64_t>(u.t0 / kW4Tokens) * a.steps * x_block(kW4Tokens, G) +
                                     static_cast<int64_t>(u.step0) * block,
                                 bytes, full_x);
                    ++x_copies;
                }
            }
        }
        return;
    }

    if (warp == kW4Consumers + 1) {             // flush
        uint32_t phase = 0;
        asm volatile("griddepcontrol.wait;" ::: "memory");
        for (int i = u0; i < u1; ++i, phase ^= 1) {
            const W4Unit u(a, i);
            if (!__all_sync(0xffffffffu, arrived(full_r, phase, w))) {
                report_timeout(w, 1, kMaxStages, phase);
                abort_flag = 1;
                return;
            }
            // lane: four rows of q, every other row of x
            const int n = (lane & 15) * 4;
            const int64_t n0 = static_cast<int64_t>(u.block) * kW4Rows + n;
#pragma unroll 1
            for (int t = lane >> 4; t < u.tokens; t += 2) {
                const float4 lo = *reinterpret_cast<const float4 *>(&red[0][t][n]);
                const float4 hi = *reinterpret_cast<const float4 *>(&red[1][t][n]);
                const float4 y = make_float4(lo.x + hi.x, lo.y + hi.y, lo.z + hi.z, lo.w + hi.w);
                if (a.slices == 1)
                    store_y(a, u.t0 + t, n0, y);
                else
                    *reinterpret_cast<float4 *>(a.partial + (static_cast<int64_t>(u.t0 + t) * a.slices + u.slice) * a.blocks * kW4Rows + n0) = y;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_r);
        }
        return;
    }

    if (warp > kW4Consumers) {                  // staging warps
        constexpr int kAhead = G == 32 ? 2 : 4;   // steps loaded ahead
        const int local = static_cast<int>(threadIdx.x) - 32 * (kW4Consumers + 2);
        RowScales<G> r[kAhead];
        // two walks over the same steps: one loads, the other stores kAhead steps later
        int li = u0, ls = 0, le = 0;
        int64_t lrow = 0;
        if (li < u1) {
            const W4Unit u(a, li);
            ls = u.step0, le = u.step1, lrow = static_cast<int64_t>(u.block) * kW4Rows + local;
        }
        auto load_next = [&](RowScales<G> &into) {
            if (li >= u1) return;
            into.load(a, lrow, static_cast<int64_t>(ls) * Step::kGroups);
            if (++ls == le && ++li < u1) {
                const W4Unit u(a, li);
                ls = u.step0, le = u.step1, lrow = static_cast<int64_t>(u.block) * kW4Rows + local;
            }
        };
#pragma unroll
        for (int k = 0; k < kAhead; ++k) load_next(r[k]);
        uint32_t stage = 0, phase = 1;
        int i = u0, s = 0, e = 0;
        int64_t row = 0;
        if (i < u1) {
            const W4Unit u(a, i);
            s = u.step0, e = u.step1, row = static_cast<int64_t>(u.block) * kW4Rows + local;
        }
        while (i < u1) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (i >= u1) break;
                // (a warp goes on, or gives up, as one)
                if (!__all_sync(0xffffffffu, arrived(empty + 8 * stage, phase, w))) {
                    report_timeout(w, 0, stage, phase);
                    abort_flag = 1;
                    return;
                }
                r[k].store(a, row, static_cast<int64_t>(s) * Step::kGroups, local,
                           reinterpret_cast<uint2 *>(ring + stage * Step::kStage + kW4QBytes));
                mbar_arrive(full + 8 * stage);
                if (++stage == kStages) stage = 0, phase ^= 1;
                load_next(r[k]);
                if (++s == e && ++i < u1) {
                    const W4Unit u(a, i);
                    s = u.step0, e = u.step1, row = static_cast<int64_t>(u.block) * kW4Rows + local;
                }
            }
        }
        return;
    }

    // consumers: rows 16 (warp % 4) .. of the unit, half warp / 4 of a step's columns
    const int half = warp >> 2, rows = (warp & 3) * 16;
    // ldmatrix: lane l gives the address of row l % 16 of chunk l / 16
    const int lrow = rows + (lane & 15);
    const uint32_t lbase = smem_u32(ring) + half * kW4BoxBytes + static_cast<uint32_t>(lrow) * 128u;
    const uint32_t lchunk = static_cast<uint32_t>(lane >> 4), lswz = static_cast<uint32_t>(lrow & 7);
    constexpr int kHalfGroups = Step::kGroups / 2;
    uint32_t stage = 0, phase = 0, rphase = 1, xphase = 0;
    const Nibbles nib;
    int staged = -1;                        // slice (of eight rows of x) in xbuf
    bool alive = true;                          // no wait of this warp has run out
    for (int i = u0; i < u1; ++i) {
        const W4Unit u(a, i);
        if (i / a.blocks != staged) {
            // done with the last slice's x (every warp arrives, also one whose wait has run out)
            if (staged >= 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(empty_x);
            }
            staged = i / a.blocks;
            if (alive && !__all_sync(0xffffffffu, arrived(full_x, xphase, w))) {
                report_timeout(w, 1, kStages, xphase);
                abort_flag = 1;
                alive = false;
            }
            xphase ^= 1;
        }
        const int tok = lane >> 2 < u.tokens ? lane >> 2 : u.tokens - 1, block = x_block(u.tokens, G);
        const unsigned char *xs = xbuf;
        float acc[4] = {};
        for (int s = u.step0; s < u.step1 && alive; ++s) {
            if (!__all_sync(0xffffffffu, arrived(full + 8 * stage, phase, w))) {
                report_timeout(w, 1, stage, phase);
                abort_flag = 1;
                alive = false;
                break;
            }
            const uint32_t q = lbase + stage * Step::kStage;
            const uint4 *x = reinterpret_cast<const uint4 *>(xs + tok * kXPitch) + (lane & 3) + half * 32;
            const float2 *m = reinterpret_cast<const float2 *>(xs + u.tokens * kXPitch) + half * kHalfGroups * 4 +
                              (lane & 3);
            const uint4 *scales =
                reinterpret_cast<const uint4 *>(ring + stage * Step::kStage + kW4QBytes) +
                half * kHalfGroups * (kW4Rows / 2) + rows / 2 + (lane >> 2);
            uint32_t v[4][4];
#pragma unroll
            for (int c = 0; c < 4; ++c) ldmatrix_x4(v[c], q + ((2u * c + lchunk) ^ lswz) * 16u);
            float p[4], p2[4], sl, sh;
            __half2 zl, zh, zl64, zh64;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const int k = c * 32;
                const uint4 b = x[4 * c];
                if (k % G == 0) {
                    const uint4 s = scales[k / G * (kW4Rows / 2)];
                    sl = __uint_as_float(s.x);
                    sh = __uint_as_float(s.z);
                    zl = as_half2(s.y);
                    zh = as_half2(s.w);
                    zl64 = __hsub2(as_half2(0x63806380u), zl);   // 960 - (1024 + z)
                    zh64 = __hsub2(as_half2(0x63806380u), zh);
                }
                const uint32_t lo = v[c >> 1][2 * (c & 1)], hi = v[c >> 1][2 * (c & 1) + 1];
                const uint32_t lo8 = lo >> 8, hi8 = hi >> 8;
                const uint32_t a0 = nib.lower(lo, zl), a1 = nib.lower(hi, zh);
                const uint32_t a2 = nib.upper(lo, zl64), a3 = nib.upper(hi, zh64);
                const uint32_t a4 = nib.lower(lo8, zl), a5 = nib.lower(hi8, zh);
                const uint32_t a6 = nib.upper(lo8, zl64), a7 = nib.upper(hi8, zh64);
                if (k % G == 0) {
                    mma_f16<true>(p, a0, a1, a2, a3, b.x, b.y);
                    mma_f16<true>(p2, a4, a5, a6, a7, b.z, b.w);
                } else {
                    mma_f16<false>(p, a0, a1, a2, a3, b.x, b.y);
                    mma_f16<false>(p2, a4, a5, a6, a7, b.z, b.w);
                }
                if ((k + 32) % G != 0) continue;
                const float2 f = m[k / G * 4];
                const float f0l = f.x * sl, f1l = f.y * sl, f0h = f.x * sh, f1h = f.y * sh;
                acc[0] += (p[0] + p2[0]) * f0l;
                acc[1] += (p[1] + p2[1]) * f1l;
                acc[2] += (p[2] + p2[2]) * f0h;
                acc[3] += (p[3] + p2[3]) * f1h;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * stage);
            if (++stage == kStages) stage = 0, phase ^= 1;
            xs += block;
        }
        if (alive && !__all_sync(0xffffffffu, arrived(empty_r, rphase, w))) {
            report_timeout(w, 1, kMaxStages, rphase);
            abort_flag = 1;
            alive = false;
        }
        if (!alive) continue;
        const int n = rows + (lane >> 2), t = 2 * (lane & 3);
        red[half][t][n] = acc[0];
        red[half][t + 1][n] = acc[1];
        red[half][t][n + 8] = acc[2];
        red[half][t + 1][n + 8] = acc[3];
        __syncwarp();
        if (lane == 0) mbar_arrive(full_r);
        rphase ^= 1;
    }
}

bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

uintptr_t type_bytes(int dtype) { return dtype == MBT_F32 ? 4 : dtype == MBT_E4M3 ? 1 : 2; }

__global__ void mbt_w4_zero_kernel(void *out, int dtype, int64_t N, int64_t ld) {
    for (int64_t n = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; n < N;
         n += static_cast<int64_t>(gridDim.x) * blockDim.x)
        store_any(out, dtype, blockIdx.y * ld + n, 0.f);
}

// The slices' sums of four outputs a thread, in slice order.
__global__ void __launch_bounds__(128) mbt_w4_slices_kernel(const W4Args a) {
    const int64_t n = (blockIdx.x * 128ll + threadIdx.x) * 4, t = blockIdx.y, pitch = static_cast<int64_t>(a.blocks) * kW4Rows;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (n >= a.N) return;
    const float *part = a.partial + t * a.slices * pitch + n;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int c = 0; c < a.slices; ++c) {
        const float4 v = *reinterpret_cast<const float4 *>(part + c * pitch);
        y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
    }
    store_y(a, t, n, y);
}

// Shared memory of a unit's part of x, with its factors.
int64_t x_bytes(int64_t steps, int rows, int group) { return steps * x_block(rows, group); }

template <int G>
cudaError_t launch_w4(const CUtensorMap &map, const W4Args &a, int grid, cudaStream_t stream) {
    constexpr int kFixed = kSwizzleAtomBytes + W4Step<G>::kStages * W4Step<G>::kStage;
    const int smem = kFixed + static_cast<int>(x_bytes(a.slice_steps, a.x_rows, G));
    static std::atomic<bool> raised[64];   // per device: the kernel's shared-memory limit is set
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !raised[dev].load(std::memory_order_relaxed)) {
        e = cudaFuncSetAttribute(mbt_w4_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kFixed + kW4XBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) raised[dev].store(true, std::memory_order_relaxed);
    }
    const dim3 units(static_cast<unsigned>((a.steps * (kW4Step / 8) + kW4XThreads - 1) / kW4XThreads),
                     static_cast<unsigned>(a.T));
    e = launch_grid(mbt_w4_x_kernel<G>, units, kW4XThreads, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pipeline(mbt_w4_kernel<G>, grid, kW4Threads, smem, stream, map, a);
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
    // The call for the first half of the rows, in whole eights, and for the others.
    auto in_halves = [&]() {
        const int64_t first = token_blocks / 2 * kW4Tokens;
        const int64_t xg = x_group ? (K + x_group - 1) / x_group : 1;
        const int rc = tile_w4_matvec(x, x_scales, q, scales, zeros, out, first, N, K, ld_x, ld_q, ld_out, group,
                                      x_group, dtype, scale_dtype, out_dtype, stream);
        if (rc != MBT_OK) return rc;
        return tile_w4_matvec(static_cast<const char *>(x) + first * ld_x * static_cast<int64_t>(type_bytes(dtype)),
                              x_scales ? x_scales + first * xg : nullptr, q, scales, zeros,
                              static_cast<char *>(out) + first * ld_out * static_cast<int64_t>(type_bytes(out_dtype)),
                              T - first, N, K, ld_x, ld_q, ld_out, group, x_group, dtype, scale_dtype, out_dtype,
                              stream);
    };
    if (T > 65535) return in_halves();   // (a grid's second dimension)
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
    const int64_t xe = static_cast<int64_t>(type_bytes(dtype));
    if (few_pays(T, N, K) && aligned(x, 16) && (T == 1 || ld_x * xe % 16 == 0)) {
        a.q = q;
        a.ld_q = ld_q;
        a.group_shift = group == 32 ? 5 : group == 64 ? 6 : 7;
        a.few_split = K <= kFewChunk ? 1 : K <= 2 * kFewChunk ? 2 : kFewWarps;
        const int64_t rows = kFewRows * (kFewWarps / a.few_split);
        const dim3 grid(static_cast<unsigned>((N + rows - 1) / rows));
        const cudaError_t e = dtype == MBT_F16    ? launch_few<MBT_F16>(a, grid, st)
                              : dtype == MBT_BF16 ? launch_few<MBT_BF16>(a, grid, st)
                                                  : launch_few<MBT_E4M3>(a, grid, st);
        return e == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
    }
    // a step's scales of a row as vectors: whole ones, aligned in every row
    const int vec = std::min(kW4Step / group, 8);
    a.vec_scales = scale_dtype != MBT_F32 && a.groups % vec == 0 && aligned(scales, 2 * static_cast<uintptr_t>(vec));
    a.vec_zeros = a.groups % 4 == 0 && aligned(zeros, 4);
    const uintptr_t xb = type_bytes(dtype);
    a.vec_x = aligned(x, 8 * xb) && (T == 1 || ld_x * static_cast<int64_t>(xb) % (8 * static_cast<int64_t>(xb)) == 0);
    a.x_rows = static_cast<int32_t>(std::min<int64_t>(T, kW4Tokens));
    const int64_t blocks = (N + kW4Rows - 1) / kW4Rows;
    a.blocks = static_cast<int32_t>(blocks);
    const int64_t steps = (K + kW4Step - 1) / kW4Step, ctas = 2 * sms;
    // Slices of K: at least as many as x's part of shared memory asks for; among
    // the counts up to four times that (or one per step, or a unit for each CTA),
    // the one with the least time for the busiest CTA, counted in steps, a unit
    // costing 0.3 of a step beside its own (8 rows of x: with nothing for a unit
    // 16384 x 16384 takes 51.9 us instead of 38.2 and 8192 x 8192 17.6 instead of 16.2;
    // with two steps 4096 x 14336 takes 16.7 instead of 15.4).
    int64_t longest = 1;
    while (longest < steps && x_bytes(longest + 1, a.x_rows, group) <= kW4XBytes)
        ++longest;
    const int64_t fewest = (steps + longest - 1) / longest;
    const int64_t most = std::min(steps, std::max(4 * fewest, ctas / (blocks * token_blocks)));
    int64_t best = -1, slices = fewest;
    for (int64_t s = fewest; s <= most; ++s) {
        const int64_t units = token_blocks * blocks * s;
        const int64_t cost = (units + ctas - 1) / ctas * (10 * ((steps + s - 1) / s) + 3);
        if (best < 0 || cost < best) best = cost, slices = s;
    }
    a.slices = static_cast<int32_t>(slices);
    a.slice_steps = static_cast<int32_t>((steps + slices - 1) / slices);
    a.steps = static_cast<int32_t>(steps);
    if (token_blocks * slices * blocks > 0x7fffffff) return MBT_ERR_UNSUPPORTED;
    a.units = static_cast<int32_t>(token_blocks * slices * blocks);
    // workspace: x as B elements, then the slices' sums
    const int64_t xb_bytes = (token_blocks * steps * x_block(kW4Tokens, group) + 255) / 256 * 256;
    const int64_t sum_bytes = slices > 1 ? slices * T * blocks * kW4Rows * 4 : 0;
    // many rows of x would take gigabytes (4096 against 16384 x 16384: 2.1 GiB), and
    // gain nothing from being one launch
    if (xb_bytes + sum_bytes > kW4MostScratch && token_blocks > 1) return in_halves();
    void *scratch = nullptr;
    WorkspaceHold hold;
    rc = hold.scratch(stream, static_cast<size_t>(xb_bytes + sum_bytes), &scratch);
    if (rc != MBT_OK) return rc;
    a.xb = static_cast<unsigned char *>(scratch);
    a.partial = reinterpret_cast<float *>(a.xb + xb_bytes);
    alignas(64) CUtensorMap map;
    rc = encode_bytes_map(&map, q, N, K / 2, ld_q, kW4Rows);
    if (rc != MBT_OK) return rc;
    const int grid = static_cast<int>(std::min<int64_t>(a.units, ctas));
    const cudaError_t e = group == 32   ? launch_w4<32>(map, a, grid, st)
                          : group == 64 ? launch_w4<64>(map, a, grid, st)
                                        : launch_w4<128>(map, a, grid, st);
    if (e != cudaSuccess) return MBT_ERR_CUDA;
    if (a.slices > 1) {
        const dim3 sums(static_cast<unsigned>((N + 511) / 512), static_cast<unsigned>(T));
        if (launch_grid(mbt_w4_slices_kernel, sums, 128, st, a) != cudaSuccess) return MBT_ERR_CUDA;
    }
    return MBT_OK;
}
