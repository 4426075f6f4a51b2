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
// Both read and write every byte once: device memory bounds them.  The scales lie in
// tiles of 128 rows x 4 blocks, the order in which the product's tensor instructions
// take them; a warp therefore works on rows r, r + 32, r + 64, r + 96 of a tile, for two
// neighbouring r, by 4 blocks: its 32 scale bytes are one aligned sector.
#include <algorithm>

#include "mbtile_elem.cuh"
#include "mbtile_layer.h"
#include "mbtile_mx4.cuh"

namespace mbt {
namespace {

constexpr int kMx4Warps = 8;

struct Mx4Args {
    const void *x;           // quantise: in; dequantise: out
    uint8_t *q, *s;
    const float *ts;
    int64_t M, K, ld_x, ld_q;
    int64_t tiles, groups;   // scale tiles of a row of tiles, eights of rows
    int32_t dtype;
    int32_t vec;             // rows of x are whole aligned 16-byte chunks
};

// The place of a lane: its row, and its block of the warp's four.
struct Mx4Place {
    int64_t row, block, scale;   // scale: byte offset
    bool in;                     // one of the scales'
    __device__ __forceinline__ Mx4Place(const Mx4Args &a) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int64_t tile = static_cast<int64_t>(blockIdx.x) * kMx4Warps + warp;   // of the row's tiles
        const int64_t group = blockIdx.y + static_cast<int64_t>(gridDim.y) * blockIdx.z;   // of 8 rows
        const int r = static_cast<int>(group & 15) * 2 + (lane >> 4), band = lane >> 2 & 3;
        row = (group >> 4) * 128 + band * 32 + r;
        block = tile * 4 + (lane & 3);
        scale = ((group >> 4) * a.tiles + tile) * 512 + r * 16 + band * 4 + (lane & 3);
        in = tile < a.tiles && group < a.groups;
    }
};

// 16 elements of a row from column j on, two to a register pair.
template <int DT>
__device__ __forceinline__ void load16(const Mx4Args &a, int64_t row, int64_t j, float (&f)[16]) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    const T *p = static_cast<const T *>(a.x) + row * a.ld_x + j;
    if (a.vec) {
        uint4 v[16 / V];
#pragma unroll
        for (int k = 0; k < 16 / V; ++k) v[k] = __ldg(reinterpret_cast<const uint4 *>(p) + k);
#pragma unroll
        for (int k = 0; k < 16 / V; ++k) {
            float g[V];
            unpack<DT>(v[k], g);
#pragma unroll
            for (int e = 0; e < V; ++e) f[k * V + e] = g[e];
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = Elem<DT>::widen(p[e]);
}

// The 16 codes of f / d; plain: with the division itself, for quotients that the
// corrected product below would not take within fp32's range.
__device__ __forceinline__ uint2 codes16(const float (&f)[16], float d, bool plain) {
    uint32_t w[2];
    const Divisor by(d);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float y[8];
        if (plain) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = -__fdiv_rn(f[8 * h + e], d);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 m = by.minus(f[8 * h + e], f[8 * h + e + 1]);
                y[e] = m.x, y[e + 1] = m.y;
            }
        }
        w[h] = to_e2m1x8(y) ^ 0x88888888u;
    }
    return make_uint2(w[0], w[1]);
}

// A lane holds a block: 16 elements, or 32 in two halves.
template <int DT, int BLOCK>
__global__ void __launch_bounds__(32 * kMx4Warps) mbt_mx4_quantize_kernel(const Mx4Args a) {
    const Mx4Place at(a);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!at.in) return;
    const int64_t j = at.block * BLOCK;
    uint32_t code = 0;
    if (at.row < a.M && j < a.K) {
        float f[BLOCK / 16][16];
        uint32_t amax = 0;
#pragma unroll
        for (int h = 0; h < BLOCK / 16; ++h) load16<DT>(a, at.row, j + 16 * h, f[h]);
#pragma unroll
        for (int h = 0; h < BLOCK / 16; ++h) amax = magnitude_max(amax, f[h]);
        const float most = __uint_as_float(amax);
        float d;
        if constexpr (BLOCK == 16) {
            const float ts = a.ts ? *a.ts : 1.f;
            // (infinity and NaN: a NaN scale)
            code = amax < 0x7f800000u ? to_e4m3x2(__fdiv_rn(most, a.ts ? 6.f * ts : 6.f), 0.f) & 0xffu : 0x7fu;
            d = Elem<MBT_F16>::widen2(e4m3x2_to_half2(code)).x * ts;
        } else {
            // the exponent of a power of two is its code; below 2^-125 that of the scale is 0
            code = amax < 0x7f800000u ? static_cast<uint32_t>(max(static_cast<int>(amax >> 23) - 2, 0)) : 0xffu;
            d = code ? __uint_as_float(code << 23) : 5.87747175e-39f;   // 2^-127
        }
        const bool none = !(d > 0.f) || amax == 0 || amax >= 0x7f800000u;   // codes 0
        const bool plain = !(most < 64.f * d) || d < 1e-30f || d > 1e30f;
        uint2 w[BLOCK / 16];
#pragma unroll
        for (int h = 0; h < BLOCK / 16; ++h) w[h] = none ? make_uint2(0u, 0u) : codes16(f[h], d, plain);
        uint8_t *q = a.q + at.row * a.ld_q + j / 2;
        if constexpr (BLOCK == 16)
            *reinterpret_cast<uint2 *>(q) = w[0];
        else
            *reinterpret_cast<uint4 *>(q) = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
    }
    a.s[at.scale] = static_cast<uint8_t>(code);
}

template <int DT, int BLOCK>
__global__ void __launch_bounds__(32 * kMx4Warps) mbt_mx4_dequantize_kernel(const Mx4Args a) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    const Mx4Place at(a);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t j = at.block * BLOCK;
    if (!at.in || at.row >= a.M || j >= a.K) return;
    const uint32_t code = a.s[at.scale];
    float s, ts = 1.f;
    if constexpr (BLOCK == 16) {
        s = Elem<MBT_F16>::widen2(e4m3x2_to_half2(code)).x;
        if (a.ts) ts = *a.ts;
    } else {
        s = code == 0xffu ? __uint_as_float(0x7fc00000u) : code ? __uint_as_float(code << 23) : 5.87747175e-39f;
    }
    const uint8_t *q = a.q + at.row * a.ld_q + j / 2;
    uint32_t w[BLOCK / 8];
    if constexpr (BLOCK == 16) {
        const uint2 v = *reinterpret_cast<const uint2 *>(q);
        w[0] = v.x, w[1] = v.y;
    } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(q);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
    T *p = static_cast<T *>(const_cast<void *>(a.x)) + at.row * a.ld_x + j;
#pragma unroll
    for (int h = 0; h < BLOCK / 8; ++h) {
        float f[8];
        uint32_t pair[4];
        e2m1x8_to_half2(w[h], pair);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 v = Elem<MBT_F16>::widen2(pair[e / 2]);
            f[e] = v.x * s * ts;
            f[e + 1] = v.y * s * ts;
        }
        if (a.vec) {
#pragma unroll
            for (int k = 0; k < 8 / V; ++k) {
                float g[V];
#pragma unroll
                for (int e = 0; e < V; ++e) g[e] = f[k * V + e];
                reinterpret_cast<uint4 *>(p + 8 * h)[k] = pack<DT>(g);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[8 * h + e] = Elem<DT>::round(f[e]);
        }
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
    // 16 groups of 8 rows to a row of tiles; a grid's second dimension holds 65535
    const int64_t groups = (M + 127) / 128 * 16, deep = (groups + 32767) / 32768;
    Mx4Args a{x, q, scales, ts, M, K, ld_x, ld_q, mx4_tiles(K, block), groups, dtype, 0};
    a.vec = aligned(x, 16) && ld_x * static_cast<int64_t>(es) % 16 == 0;
    const dim3 grid(static_cast<unsigned>((a.tiles + kMx4Warps - 1) / kMx4Warps),
                    static_cast<unsigned>(deep > 1 ? 32768 : groups), static_cast<unsigned>(deep));
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
