// Internal interface of the layer operators' translation units.
#pragma once

#include "internal.h"

namespace mbt {

struct NormArgs {
    const void *x, *res, *w;
    void *out, *res_out;
    float *scales, *rstd;
    int64_t M, N, ld_x, ld_res, ld_out, ld_res_out;
    int64_t groups;          // scales per row
    int32_t wdt, quant;      // quant: -1 none, 0 a scale per row, else columns per scale
    float eps, woff;
};

struct NormGradArgs {
    const void *dy, *h, *w, *dres;
    const float *rstd;
    void *dx;
    float *dw, *partial;     // partial: [splits][N]
    int64_t M, N, ld_dy, ld_h, ld_dres, ld_dx;
    int64_t splits;
    int32_t wdt;
    float woff;
};

// Layer norm: as above, with a mean, a bias and its gradient.
struct LayerNormArgs {
    const void *x, *res, *w, *b;
    void *out, *res_out;
    float *scales, *mean, *rstd;
    int64_t M, N, ld_x, ld_res, ld_out, ld_res_out;
    int64_t groups;
    int32_t wdt, quant;      // wdt: of weight and bias
    float eps, woff;
};

struct LayerNormGradArgs {
    const void *dy, *h, *w, *dres;
    const float *mean, *rstd;
    void *dx;
    float *dw, *db, *partial;   // partial: [2][splits][N], dw's and then db's
    int64_t M, N, ld_dy, ld_h, ld_dres, ld_dx;
    int64_t splits;
    int32_t wdt;
    float woff;
};

// (mbtile_layernorm_f16.cu, _bf16.cu, _f32.cu)  The calls after their checks, M > 0 (the gradient: N > 0 too).
template <int DT>
cudaError_t layernorm_forward(const LayerNormArgs &a, cudaStream_t s);
template <int DT>
int layernorm_backward(const LayerNormGradArgs &a, cudaStream_t s);

// (mbtile_norm_f16.cu, _bf16.cu, _f32.cu)  The calls after their checks, M > 0 (the gradient: N > 0 too).
template <int DT>
cudaError_t norm_forward(const NormArgs &a, cudaStream_t s);
template <int DT>
int norm_backward(const NormGradArgs &a, cudaStream_t s);

// (mbtile_host.cpp)  2-D tiled map over `rows` rows of `row_bytes` bytes, `ld`
// bytes apart: box = 128 bytes x box_rows rows, 128-byte swizzle, zero fill.
int encode_bytes_map(CUtensorMap *map, const void *src, int64_t rows, int64_t row_bytes, int64_t ld,
                     int box_rows);
// (mbtile_host.cpp)  3-D tiled map over `row_tiles` x `tiles` tiles of 512 bytes, one after
// the other: box = `box` tiles of a row of tiles, zero fill.
int encode_scales_map(CUtensorMap *map, const void *src, int64_t row_tiles, int64_t tiles, int box);
// (mbtile_host.cpp)  Address of the current device's status word, looked up once per device.
int device_status_word(int32_t **word);

// Launch of any grid with programmatic stream serialization; the kernel waits for
// its predecessor itself.
template <class K, class A>
cudaError_t launch_grid(K kernel, dim3 grid, int threads, cudaStream_t stream, const A &a) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace mbt
