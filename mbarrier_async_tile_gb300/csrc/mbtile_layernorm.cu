// tile_layernorm and tile_layernorm_backward: layer norm over a matrix's rows, with the
// residual's addition, and its gradient.
//
//   h = x + r    mu_i = mean_j h_ij    rstd_i = (mean_j (h_ij - mu_i)^2 + eps)^(-1/2)
//   xh = (h - mu) rstd    y = xh (w + o) + b    g = dy (w + o)
//   dx = rstd (g - mean_j g - xh mean_j(g xh)) + dres    dw_j = sum_i dy xh    db_j = sum_i dy
//
// Both compute a handful of operations per element, and device memory bounds them.  The norm,
// and the gradient of rows that the shared-memory ring takes, read and write every matrix once;
// the gradient of longer rows reads dy and h for dw and db and again for dx.  All sums are
// fp32.  The kernels are in mbtile_layernorm.cuh; here are the entry points and their checks.
#include "mbtile_layer.h"

namespace mbt {
namespace {

bool float_type(int dtype) { return dtype == MBT_F16 || dtype == MBT_BF16 || dtype == MBT_F32; }

bool aligned_elem(const void *p, int dtype) {
    return reinterpret_cast<uintptr_t>(p) % (dtype == MBT_F32 ? 4u : 2u) == 0;
}

constexpr int64_t kMaxIndex = int64_t{1} << 46;   // elements an address may be away

// Row pitch (0 => N) and its bounds.
bool pitch(int64_t *ld, int64_t M, int64_t N) {
    if (*ld == 0) *ld = N;
    return *ld >= N && (M == 0 || *ld <= kMaxIndex / M);
}

}  // namespace
}  // namespace mbt

extern "C" int tile_layernorm(const void *x, const void *residual, const void *weight, const void *bias, void *out,
                              void *residual_out, float *scales, float *mean, float *rstd, int64_t M, int64_t N,
                              int64_t ld_x, int64_t ld_res, int64_t ld_out, int64_t ld_res_out, int dtype,
                              int weight_dtype, int quant, float eps, float weight_offset, void *stream) {
    using namespace mbt;
    if (M < 0 || N < 0 || N > 0x7fffffff || !float_type(dtype) || (weight && !float_type(weight_dtype)) ||
        (bias && !weight) || !(eps >= 0.f))
        return MBT_ERR_ARG;
    if (quant != MBT_QUANT_NONE && quant != MBT_QUANT_ROW && quant != 32 && quant != 64 && quant != 128)
        return MBT_ERR_UNSUPPORTED;
    if (!pitch(&ld_x, M, N) || !pitch(&ld_res, M, N) || !pitch(&ld_out, M, N) || !pitch(&ld_res_out, M, N))
        return MBT_ERR_ARG;
    if (M == 0) return MBT_OK;
    if (!mean || !rstd || (N > 0 && (!x || !out)) || (quant != MBT_QUANT_NONE) != (scales != nullptr) ||
        (residual_out && !residual))
        return MBT_ERR_ARG;
    if (!aligned_elem(x, dtype) || !aligned_elem(residual, dtype) || !aligned_elem(residual_out, dtype) ||
        (weight && (!aligned_elem(weight, weight_dtype) || !aligned_elem(bias, weight_dtype))) ||
        (quant == MBT_QUANT_NONE && !aligned_elem(out, dtype)) || !aligned_elem(mean, MBT_F32) ||
        !aligned_elem(rstd, MBT_F32) || !aligned_elem(scales, MBT_F32))
        return MBT_ERR_ALIGN;
    const LayerNormArgs a{x,      residual, weight, bias,       out,  residual_out,
                          scales, mean,     rstd,   M,          N,    ld_x,
                          ld_res, ld_out,   ld_res_out, quant > 0 ? (N + quant - 1) / quant : 1, weight_dtype,
                          quant,  eps,      weight_offset};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == MBT_F16    ? layernorm_forward<MBT_F16>(a, s)
                          : dtype == MBT_BF16 ? layernorm_forward<MBT_BF16>(a, s)
                                              : layernorm_forward<MBT_F32>(a, s);
    return e == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
}

extern "C" int tile_layernorm_backward(const void *dy, const void *h, const float *mean, const float *rstd,
                                       const void *weight, const void *dresidual, void *dx, float *dweight,
                                       float *dbias, int64_t M, int64_t N, int64_t ld_dy, int64_t ld_h, int64_t ld_dres,
                                       int64_t ld_dx, int dtype, int weight_dtype, float weight_offset, void *stream) {
    using namespace mbt;
    if (M < 0 || N < 0 || N > 0x7fffffff || !float_type(dtype) || (weight && !float_type(weight_dtype)))
        return MBT_ERR_ARG;
    if (!pitch(&ld_dy, M, N) || !pitch(&ld_h, M, N) || !pitch(&ld_dres, M, N) || !pitch(&ld_dx, M, N))
        return MBT_ERR_ARG;
    if (N == 0) return MBT_OK;
    if (M > 0 && (!dy || !h || !mean || !rstd || !dx)) return MBT_ERR_ARG;
    if (!aligned_elem(dy, dtype) || !aligned_elem(h, dtype) || !aligned_elem(dresidual, dtype) ||
        !aligned_elem(dx, dtype) || (weight && !aligned_elem(weight, weight_dtype)) || !aligned_elem(mean, MBT_F32) ||
        !aligned_elem(rstd, MBT_F32) || !aligned_elem(dweight, MBT_F32) || !aligned_elem(dbias, MBT_F32))
        return MBT_ERR_ALIGN;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) {
        for (float *d : {dweight, dbias})
            if (d && cudaMemsetAsync(d, 0, static_cast<size_t>(N) * 4, s) != cudaSuccess) return MBT_ERR_CUDA;
        return MBT_OK;
    }
    const LayerNormGradArgs a{dy, h, weight, dresidual, mean, rstd, dx, dweight, dbias, nullptr, M, N, ld_dy, ld_h,
                              ld_dres, ld_dx, 1, weight_dtype, weight_offset};
    return dtype == MBT_F16    ? layernorm_backward<MBT_F16>(a, s)
           : dtype == MBT_BF16 ? layernorm_backward<MBT_BF16>(a, s)
                               : layernorm_backward<MBT_F32>(a, s);
}
