// tile_w4_matvec: products of a few rows of activations with a matrix held in
// 4 bits, y[t, n] = sum_k x[t, k] (q[n, k] - z[n, k / g]) s[n, k / g].
#include <algorithm>

#include "internal.h"
#include "mbtile_elem.cuh"
#include "mbtile_ptx.cuh"

namespace mbt {
namespace {

struct W4Args {
    const void *x;
    const uint8_t *q;
    const void *s;
    const uint8_t *z;
    const float *xs;
    void *out;
    int64_t T, N, K, ld_x, ld_q, ld_out;
    int64_t groups, x_groups;   // scales of a row of q, of a row of x
    int32_t group, x_group;     // columns a scale covers
    int32_t xdt, sdt, odt;
};

__device__ __forceinline__ float x_at(const W4Args &a, int64_t t, int64_t k) {
    if (a.xdt != MBT_E4M3) return load_any(a.x, a.xdt, t * a.ld_x + k);
    const uint8_t c = static_cast<const uint8_t *>(a.x)[t * a.ld_x + k];
    return Elem<MBT_F16>::widen2(e4m3x2_to_half2(c)).x * a.xs[t * a.x_groups + k / a.x_group];
}

constexpr int kW4Threads = 256;
constexpr int kW4Tokens = 8;

// A warp per row of q and eight tokens.
__global__ void __launch_bounds__(kW4Threads) mbt_w4_rows_kernel(const W4Args a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t n = static_cast<int64_t>(blockIdx.x) * (kW4Threads / 32) + (threadIdx.x >> 5);
    const int64_t t0 = static_cast<int64_t>(blockIdx.y) * kW4Tokens;
    if (n >= a.N) return;
    float acc[kW4Tokens] = {};
    for (int64_t k = lane * 8; k < a.K; k += 256) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(a.q + n * a.ld_q + k / 2);
        const int64_t g = n * a.groups + k / a.group;
        const float s = load_any(a.s, a.sdt, g);
        const float z = a.z ? static_cast<float>(a.z[g]) : 8.f;
#pragma unroll
        for (int t = 0; t < kW4Tokens; ++t) {
            if (t0 + t >= a.T) break;
            float p = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                p += x_at(a, t0 + t, k + i) * (static_cast<float>(w >> (4 * i) & 15u) - z);
            acc[t] += p * s;
        }
    }
#pragma unroll
    for (int t = 0; t < kW4Tokens; ++t) {
        if (t0 + t >= a.T) break;
        const float y = warp_sum(acc[t]);
        if (lane == 0) store_any(a.out, a.odt, (t0 + t) * a.ld_out + n, y);
    }
}

bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

uintptr_t type_bytes(int dtype) { return dtype == MBT_F32 ? 4 : dtype == MBT_E4M3 ? 1 : 2; }

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
    W4Args a{x, q, scales, zeros, x_scales, out, T, N, K, ld_x, ld_q, ld_out,
             (K + group - 1) / group, x_group ? (K + x_group - 1) / x_group : 1, group,
             x_group ? x_group : static_cast<int32_t>(std::max<int64_t>(K, 1)), dtype, scale_dtype,
             out_dtype};
    const int64_t tb = (T + kW4Tokens - 1) / kW4Tokens;
    if (tb > 65535) return MBT_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((N + 7) / 8), static_cast<unsigned>(tb));
    cfg.blockDim = dim3(kW4Threads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mbt_w4_rows_kernel, a) == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
}
