// tile_mx4_quantize and tile_mx4_dequantize: matrices in microscaled 4-bit floats,
// a block of a row's elements sharing an 8-bit scale (see mbtile.h for the formats).
//
//   blocks of 16:  s = e4m3(a / (6 t))   d = s t   code = e2m1(x / d)
//   blocks of 32:  s = 2^(floor(log2 a) - 2)       code = e2m1(x / s)
//
// with a the block's largest magnitude and t the tensor scale.  Every quotient is
// rounded to fp32 before it is rounded to a code, as the formulas read in fp32, so
// that codes do not depend on how a kernel divides.
//
// Both read and write every byte once: device memory bounds them.  A warp takes 32
// pieces of 16 or 32 bytes, side by side, of each of two or four rows.  (A lane with a
// block of its own reads lines that 32 lanes each touch eight times over: fp32 16384 x
// 16384 by 32 260 us, 4.7 TB/s.)  The scales lie in tiles of 128 rows x 4 blocks, the
// order in which the product's tensor instructions take them; the rows are 32 apart, so that
// their scales lie side by side.
#include <algorithm>

#include "mbtile_elem.cuh"
#include "mbtile_layer.h"
#include "mbtile_mx4.cuh"

namespace mbt {
namespace {

constexpr int kMx4Warps = 4;
// Rows of a warp.  Fewer to quantise, whose arithmetic wants the registers that more warps
// then share (fp32 16384 x 16384 by 32, us, with 2 / 4: 181 / 205; back 110 / 101).
constexpr int kQuantizeRows = 2;
constexpr int kDequantizeRows = 4;

struct Mx4Args {
    const void *x;           // quantise: in; dequantise: out
    uint8_t *q, *s;
    const float *ts;
    int64_t M, K, ld_x, ld_q;
    int64_t tiles;           // scale tiles of a row of tiles
    uint32_t chunks;         // of a warp's columns across a row
    uint32_t warps;          // chunks x their rows
    int32_t vec;             // rows of x are aligned to 16 bytes, 2: to 32
};

// A lane's place: the first of its V columns, and its warp's rows.
template <int V, int BLOCK, int ROWS>
struct Mx4Place {
    int64_t col, first;      // first: row
    int64_t tile;            // the lane's block's scale tile
    int r, band, byte;       // row in its band of 32, the first row's band; the block's byte of a row's four
    bool in, lane_in_scales; // one of the matrix's warps; its block has a byte of scale
    __device__ __forceinline__ Mx4Place(const Mx4Args &a) {
        const uint32_t id = blockIdx.x * kMx4Warps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
        in = id < a.warps;
        const uint32_t group = id / a.chunks, chunk = id - group * a.chunks;
        col = (static_cast<int64_t>(chunk) * 32 + lane) * V;
        constexpr uint32_t kGroups = 128 / ROWS;   // of a row of tiles
        const uint32_t row_tile = group / kGroups;
        r = static_cast<int>(group & 31);
        band = static_cast<int>(group % kGroups >> 5) * ROWS;
        first = static_cast<int64_t>(row_tile) * 128 + band * 32 + r;
        const int64_t block = col / BLOCK;
        tile = row_tile * a.tiles + (block >> 2);
        byte = static_cast<int>(block & 3);
        lane_in_scales = (block >> 2) < a.tiles;
    }
    __device__ __forceinline__ int64_t row(int i) const { return first + i * 32; }
    __device__ __forceinline__ int64_t scale(int i) const { return tile * 512 + r * 16 + (band + i) * 4 + byte; }
};

// 32 bytes of a row: at once, as two vectors, or by elements, as its alignment allows.
template <int DT>
__device__ __forceinline__ void load_pair(const Mx4Args &a, int64_t row, int64_t col, uint4 (&v)[2]) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    const T *p = static_cast<const T *>(a.x) + row * a.ld_x + col;
    if (a.vec == 2) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z),
                       "=r"(v[1].w)
                     : "l"(p));
    } else if (a.vec) {
        v[0] = __ldg(reinterpret_cast<const uint4 *>(p));
        v[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float f[V];
#pragma unroll
            for (int e = 0; e < V; ++e) f[e] = Elem<DT>::widen(p[h * V + e]);
            v[h] = pack<DT>(f);
        }
    }
}

// The codes of E elements f by d, eight to a word.
template <int E, int BLOCK>
__device__ __forceinline__ void codes_of(float (&f)[E], float d, float most, uint32_t (&w)[E / 8]) {
    if (BLOCK == 16 && !(most < 64.f * d)) {
        // a scale at its largest: quotients far past 6, which might leave fp32's range
        const float high = 32.f * d;
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = fminf(fmaxf(f[e], -high), high);
    }
    // (of a power of two the inverse is exact, 2^127 for 2^-127)
    const Pair inv(__uint_as_float(0x7f000000u - (__float_as_uint(d) & 0x7f800000u)));
    const Divisor by(d);
#pragma unroll
    for (int h = 0; h < E / 8; ++h) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 v = BLOCK == 32 ? (Pair(f[8 * h + e], f[8 * h + e + 1]) * inv).get()
                                         : by.minus(f[8 * h + e], f[8 * h + e + 1]);
            y[e] = v.x, y[e + 1] = v.y;
        }
        w[h] = to_e2m1x8(y) ^ (BLOCK == 32 ? 0u : 0x88888888u);
    }
}

// A lane takes 32 bytes of a row: of 16-bit elements a whole block of 16, so that the
// scale's arithmetic is done once a block.  fp32 16384 x 16384 by 32 181 us, 6.7 TB/s; bf16 16384 x
// 8192 by 16 63 us, 5.4 TB/s, bound by instructions; 2047 x 8192 10.7 us (with 16 bytes a lane
// 14.5), by the latency of a start and a few loads.
template <int DT, int BLOCK>
__global__ void __launch_bounds__(32 * kMx4Warps, 10) mbt_mx4_quantize_kernel(const Mx4Args a) {
    constexpr int V = Elem<DT>::kVec, E = 2 * V;
    const Mx4Place<E, BLOCK, kQuantizeRows> at(a);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!at.in) return;
    const float ts = BLOCK == 16 && a.ts ? *a.ts : 1.f;
    const float t = 6.f * ts, it = __frcp_rn(t);
    uint4 v[kQuantizeRows][2];
#pragma unroll
    for (int i = 0; i < kQuantizeRows; ++i) {
        v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (at.row(i) < a.M && at.col < a.K) load_pair<DT>(a, at.row(i), at.col, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kQuantizeRows; ++i) {
        float f[E];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float g[V];
            unpack<DT>(v[i][h], g);
#pragma unroll
            for (int e = 0; e < V; ++e) f[h * V + e] = g[e];
        }
        uint32_t amax = magnitude_max(0u, f);
#pragma unroll
        for (int o = 1; o < BLOCK / E; o <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float most = __uint_as_float(amax);
        const bool finite = amax < 0x7f800000u;
        uint32_t code;
        float d;
        if constexpr (BLOCK == 16) {
            // a / t; past 448 by its size alone, which also keeps the quotient in range
            const float q = most < 1024.f * t ? divide(Pair(most), Pair(-t), Pair(it)).get().x : kE4m3Max;
            code = !finite ? 0x7fu : amax ? to_e4m3x2(q, 0.f) & 0xffu : 0u;
            d = Elem<MBT_F16>::widen2(e4m3x2_to_half2(code)).x * ts;
        } else {
            // the exponent of a power of two is its code; below 2^-125 that of the scale is 0
            code = finite ? static_cast<uint32_t>(max(static_cast<int>(amax >> 23) - 2, 0)) : 0xffu;
            d = code ? __uint_as_float(code << 23) : 5.87747175e-39f;   // 2^-127
        }
        uint32_t w[E / 8] = {};
        if (d > 0.f && amax != 0 && finite) codes_of<E, BLOCK>(f, d, most, w);
        if (at.row(i) < a.M && at.col < a.K) {
            uint8_t *q = a.q + at.row(i) * a.ld_q + at.col / 2;
            if constexpr (E == 16)
                *reinterpret_cast<uint2 *>(q) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint32_t *>(q) = w[0];
        }
        if (at.lane_in_scales && at.col % BLOCK == 0) a.s[at.scale(i)] = static_cast<uint8_t>(code);
    }
}

// fp32 16384 x 16384 by 32 back to bf16 101 us, 6.7 TB/s; bf16 2047 x 8192 by 16 8.4 us, 5.1 TB/s.
template <int DT, int BLOCK>
__global__ void __launch_bounds__(32 * kMx4Warps) mbt_mx4_dequantize_kernel(const Mx4Args a) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    const Mx4Place<V, BLOCK, kDequantizeRows> at(a);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!at.in || at.col >= a.K) return;
    const float ts = BLOCK == 16 && a.ts ? *a.ts : 1.f;
    uint32_t w[kDequantizeRows], code[kDequantizeRows];
#pragma unroll
    for (int i = 0; i < kDequantizeRows; ++i) {
        w[i] = code[i] = 0;
        if (at.row(i) >= a.M) continue;
        const uint8_t *q = a.q + at.row(i) * a.ld_q + at.col / 2;
        w[i] = V == 8 ? __ldg(reinterpret_cast<const uint32_t *>(q)) : __ldg(reinterpret_cast<const uint16_t *>(q));
        code[i] = __ldg(a.s + at.scale(i));
    }
#pragma unroll
    for (int i = 0; i < kDequantizeRows; ++i) {
        if (at.row(i) >= a.M) continue;
        float s;
        if constexpr (BLOCK == 16)
            s = Elem<MBT_F16>::widen2(e4m3x2_to_half2(code[i])).x;
        else
            s = code[i] == 0xffu ? __uint_as_float(0x7fc00000u) : code[i] ? __uint_as_float(code[i] << 23) : 5.87747175e-39f;
        uint32_t pair[4];
        e2m1x8_to_half2(w[i], pair);
        float f[V];
#pragma unroll
        for (int e = 0; e < V; e += 2) {
            const float2 v = Elem<MBT_F16>::widen2(pair[e / 2]);
            f[e] = v.x * s * ts;
            f[e + 1] = v.y * s * ts;
        }
        T *p = static_cast<T *>(const_cast<void *>(a.x)) + at.row(i) * a.ld_x + at.col;
        if (a.vec)
            *reinterpret_cast<uint4 *>(p) = pack<DT>(f);
        else
#pragma unroll
            for (int e = 0; e < V; ++e) p[e] = Elem<DT>::round(f[e]);
    }
}

bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <bool BACK, int DT>
cudaError_t launch_mx4(const Mx4Args &a, int block, dim3 grid, cudaStream_t s) {
    if constexpr (BACK)
        return block == 16 ? launch_grid(mbt_mx4_dequantize_kernel<DT, 16>, grid, 32 * kMx4Warps, s, a)
                           : launch_grid(mbt_mx4_dequantize_kernel<DT, 32>, grid, 32 * kMx4Warps, s, a);
    return block == 16 ? launch_grid(mbt_mx4_quantize_kernel<DT, 16>, grid, 32 * kMx4Warps, s, a)
                       : launch_grid(mbt_mx4_quantize_kernel<DT, 32>, grid, 32 * kMx4Warps, s, a);
}

template <bool BACK>
int mx4_convert(const void *x, const float *ts, uint8_t *q, uint8_t *scales, int64_t M, int64_t K, int64_t ld_x,
                int64_t ld_q, int block, int dtype, void *stream) {
    if (M < 0 || K < 0 || M > 0x7fffffff || K > 0x7fffffff || dtype < MBT_F16 || dtype > MBT_F32) return MBT_ERR_ARG;
    if ((block != 16 && block != 32) || K % 32 != 0) return MBT_ERR_UNSUPPORTED;
    if (block != 16 && ts) return MBT_ERR_ARG;
    if (ld_x == 0) ld_x = K;
    if (ld_q == 0) ld_q = K / 2;
    if (ld_x < K || ld_q < K / 2 || ld_x > (1ll << 40) || ld_q >= (1ll << 40)) return MBT_ERR_ARG;
    if (M == 0 || K == 0) return MBT_OK;
    if (!x || !q || !scales) return MBT_ERR_ARG;
    const uintptr_t es = dtype == MBT_F32 ? 4 : 2;
    if (!aligned(x, es) || !aligned(q, 16) || ld_q % 16 != 0 || !aligned(scales, 16) || !aligned(ts, 4))
        return MBT_ERR_ALIGN;
    const int64_t wide = BACK ? 512 : 1024;   // bytes of a warp and row of x
    const int64_t chunks = (K * static_cast<int64_t>(es) + wide - 1) / wide, warps = (M + 127) / 128 * (128 / (BACK ? kDequantizeRows : kQuantizeRows)) * chunks;
    if (warps > 0xffffffffll - kMx4Warps) return MBT_ERR_UNSUPPORTED;
    Mx4Args a{x, q, scales, ts, M, K, ld_x, ld_q, mx4_tiles(K, block), static_cast<uint32_t>(chunks), static_cast<uint32_t>(warps), 0};
    const uintptr_t pitch = static_cast<uintptr_t>(ld_x) * es;
    a.vec = aligned(x, 32) && pitch % 32 == 0 ? 2 : aligned(x, 16) && pitch % 16 == 0;
    const dim3 grid(static_cast<unsigned>((warps + kMx4Warps - 1) / kMx4Warps));
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == MBT_F16    ? launch_mx4<BACK, MBT_F16>(a, block, grid, s)
                          : dtype == MBT_BF16 ? launch_mx4<BACK, MBT_BF16>(a, block, grid, s)
                                              : launch_mx4<BACK, MBT_F32>(a, block, grid, s);
    return e == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
}

}  // namespace
}  // namespace mbt

extern "C" int tile_mx4_quantize(const void *x, const float *tensor_scale, uint8_t *q, uint8_t *scales, int64_t M,
                                 int64_t K, int64_t ld_x, int64_t ld_q, int block, int dtype, void *stream) {
    return mbt::mx4_convert<false>(x, tensor_scale, q, scales, M, K, ld_x, ld_q, block, dtype, stream);
}

extern "C" int tile_mx4_dequantize(const uint8_t *q, const uint8_t *scales, const float *tensor_scale, void *out,
                                   int64_t M, int64_t K, int64_t ld_q, int64_t ld_out, int block, int out_dtype,
                                   void *stream) {
    return mbt::mx4_convert<true>(out, tensor_scale, const_cast<uint8_t *>(q), const_cast<uint8_t *>(scales), M, K,
                                  ld_out, ld_q, block, out_dtype, stream);
}

extern "C" int64_t tile_mx4_scale_bytes(int64_t M, int64_t K, int block) {
    if (M < 0 || K < 0 || M > 0x7fffffff || K > 0x7fffffff || (block != 16 && block != 32)) return MBT_ERR_ARG;
    return (M + 127) / 128 * mbt::mx4_tiles(K, block) * 512;
}
