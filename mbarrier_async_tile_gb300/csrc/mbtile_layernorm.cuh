// Kernels of tile_layernorm and tile_layernorm_backward, for one element type per
// translation unit (mbtile_layernorm_f16.cu, _bf16.cu, _f32.cu).  They share the norm's
// parts: rows in 16-byte chunks by address, rows in registers, the ring of rows in shared
// memory, the plan of a ring (mbtile_norm.cuh).
//
// The variance is summed from deviations, in a second pass over the row's elements
// where they are held: sums of squares would lose the variance of rows whose mean is
// large against it (fp32, mean 1000, deviation 1: the third digit).
#pragma once

#include "mbtile_norm.cuh"

namespace mbt {
namespace {

// Any strides and lengths, one element per access: a CTA per row, a pass for the mean, one
// for the variance, with a scale for the row one for the largest magnitude, and one that
// writes (all but the first hit the caches).
template <int DT>
__global__ void __launch_bounds__(kRowThreads) mbt_layernorm_rows_kernel(const LayerNormArgs a) {
    using T = typename Elem<DT>::type;
    __shared__ float red[2 * kRowThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t i = blockIdx.x; i < a.M; i += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + i * a.ld_x;
        const T *r = a.res ? static_cast<const T *>(a.res) + i * a.ld_res : nullptr;
        T *ro = a.res_out ? static_cast<T *>(a.res_out) + i * a.ld_res_out : nullptr;
        auto h_at = [&](int64_t j) { return Elem<DT>::widen(x[j]) + (r ? Elem<DT>::widen(r[j]) : 0.f); };
        uint32_t amax = 0;
        float sum = 0.f;
        for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads) sum += h_at(j);
        block_reduce<kRowThreads>(sum, amax, red);
        const float mean = a.N ? sum / static_cast<float>(a.N) : 0.f;
        float ss = 0.f;
        for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads) {
            const float d = h_at(j) - mean;
            ss += d * d;
        }
        block_reduce<kRowThreads>(ss, amax, red);
        const float rstd = 1.f / sqrtf((a.N ? ss / static_cast<float>(a.N) : 0.f) + a.eps);
        auto y_of = [&](float h, int64_t j) {
            return (h - mean) * rstd * weight_at(a.w, a.wdt, a.woff, j) + (a.b ? load_any(a.b, a.wdt, j) : 0.f);
        };
        if (threadIdx.x == 0) {
            a.mean[i] = mean;
            a.rstd[i] = rstd;
        }
        if (a.quant <= 0) {
            float none = 0.f;
            if (a.quant == 0) {
                for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads) amax = max(amax, magnitude(y_of(h_at(j), j)));
                block_reduce<kRowThreads>(none, amax, red);
            }
            const float scale = group_scale(amax);
            if (a.quant == 0 && threadIdx.x == 0) a.scales[i] = scale;
            for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads) {
                const float h = h_at(j), y = y_of(h, j);
                if (a.quant == 0)
                    static_cast<uint8_t *>(a.out)[i * a.ld_out + j] = static_cast<uint8_t>(to_e4m3x2(y / scale, 0.f));
                else
                    static_cast<T *>(a.out)[i * a.ld_out + j] = Elem<DT>::round(y);
                if (ro) ro[j] = Elem<DT>::round(h);
            }
            continue;
        }
        // groups of 32, 64 or 128 columns: a warp takes 128 columns at a time
        for (int64_t j0 = warp * 128; j0 < a.N; j0 += kRowThreads * 4) {
            float y[4];
            uint32_t m[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t j = j0 + 32 * k + lane;
                y[k] = 0.f;
                if (j < a.N) {
                    const float h = h_at(j);
                    y[k] = y_of(h, j);
                    if (ro) ro[j] = Elem<DT>::round(h);
                }
                m[k] = __reduce_max_sync(0xffffffffu, magnitude(y[k]));
            }
            if (a.quant >= 64) {
                m[0] = m[1] = max(m[0], m[1]);
                m[2] = m[3] = max(m[2], m[3]);
            }
            if (a.quant >= 128) m[0] = m[1] = m[2] = m[3] = max(m[0], m[2]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t j = j0 + 32 * k + lane;
                const float scale = group_scale(m[k]);
                if (j < a.N) {
                    static_cast<uint8_t *>(a.out)[i * a.ld_out + j] = static_cast<uint8_t>(to_e4m3x2(y[k] / scale, 0.f));
                    if (j % a.quant == 0) a.scales[i * a.groups + j / a.quant] = scale;
                }
            }
        }
    }
}

struct LayerNormVecArgs {
    LayerNormArgs a;
    int32_t tpr, wmode;      // threads per row (a power of two), weight access
    int32_t bmode;           // the bias's
    int32_t phased;          // rows may start inside a chunk
};

// The bias of a chunk's elements, as load_weight has the weight; none: 0.
template <int DT>
__device__ __forceinline__ void load_bias(const void *b, int mode, int wdt, int64_t p, int off, int64_t N,
                                          float (&f)[Elem<DT>::kVec]) {
    if (mode == kNoWeight) {
#pragma unroll
        for (int e = 0; e < Elem<DT>::kVec; ++e) f[e] = 0.f;
        return;
    }
    load_weight<DT>(b, mode, wdt, 0.f, p, off, N, f);
}

// `tpr` threads hold a row in registers, C chunks each: one pass over memory.
template <int DT, int C, bool RES, bool Q>
__global__ void __launch_bounds__(1024) mbt_layernorm_kernel(const __grid_constant__ LayerNormVecArgs va) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    __shared__ float red[2][32];
    __shared__ uint32_t redm[32];
    const LayerNormArgs &a = va.a;
    const int tpr = va.tpr, t = threadIdx.x & (tpr - 1);
    const int64_t i = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = i < a.M;
    const int off = va.phased ? static_cast<int>((i * a.ld_x) & (V - 1)) : 0;
    const int64_t end = live ? a.N + off : 0;          // in elements from the first chunk
    const T *x = static_cast<const T *>(a.x) + i * a.ld_x - off;
    const T *r = static_cast<const T *>(a.res) + i * a.ld_res - off;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float h[C][V];
    {
        uint4 xv[C], rv[RES ? C : 1];
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int64_t p = static_cast<int64_t>(t + k * tpr) * V;
            xv[k] = make_uint4(0, 0, 0, 0);
            if (RES) rv[k] = make_uint4(0, 0, 0, 0);
            if (p >= end) continue;
            const int lo = p < off ? off : 0, hi = end - p < V ? static_cast<int>(end - p) : V;
            xv[k] = load_chunk<DT>(x + p, lo, hi);
            if (RES) rv[k] = load_chunk<DT>(r + p, lo, hi);
        }
#pragma unroll
        for (int k = 0; k < C; ++k) {
            unpack<DT>(xv[k], h[k]);
            if (RES) {
                float f[V];
                unpack<DT>(rv[k], f);
#pragma unroll
                for (int e = 0; e < V; ++e) h[k][e] += f[e];
            }
        }
    }
    // the sum over the row, in all of its threads
    auto row_sum = [&](float v, int turn) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < tpr) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (tpr > 32) {                                // one row per CTA
            if ((t & 31) == 0) red[turn][t >> 5] = v;
            __syncthreads();
            v = warp_sum((t & 31) < (tpr >> 5) ? red[turn][t & 31] : 0.f);
        }
        return v;
    };
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) sum += h[k][e];
    const float n = static_cast<float>(a.N), mean = row_sum(sum, 0) / n;
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int64_t p = static_cast<int64_t>(t + k * tpr) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = h[k][e] - mean;
            if (p + e >= off && p + e < end) ss += d * d;
        }
    }
    const float rstd = 1.f / sqrtf(row_sum(ss, 1) / n + a.eps);
    auto y_of = [&](int k, int64_t p, float (&y)[V]) {
        float b[V];
        load_weight<DT>(a.w, va.wmode, a.wdt, a.woff, p, off, a.N, y);
        load_bias<DT>(a.b, va.bmode, a.wdt, p, off, a.N, b);
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = (h[k][e] - mean) * rstd * y[e] + b[e];
    };
    float scale = 0.f;
    Divisor by;
    if (Q && a.quant == 0) {
        uint32_t amax = 0;
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int64_t p = static_cast<int64_t>(t + k * tpr) * V;
            if (p >= end) continue;
            float y[V];
            y_of(k, p, y);
#pragma unroll
            for (int e = 0; e < V; ++e)
                if (p + e < off || p + e >= end) y[e] = 0.f;
            amax = magnitude_max(amax, y);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < tpr) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (tpr > 32) {
            if ((t & 31) == 0) redm[t >> 5] = amax;
            __syncthreads();
            amax = __reduce_max_sync(0xffffffffu, (t & 31) < (tpr >> 5) ? redm[t & 31] : 0u);
        }
        scale = group_scale(amax);
        by = Divisor(scale);
    }
    if (live && t == 0) {
        a.mean[i] = mean;
        a.rstd[i] = rstd;
        if (Q && a.quant == 0) a.scales[i] = scale;
    }
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int64_t p = static_cast<int64_t>(t + k * tpr) * V;
        if (!Q && p >= end) continue;
        const int lo = p < off ? off : 0, hi = end - p < V ? static_cast<int>(end - p) : V;
        float y[V];
        if (RES && p < end && a.res_out)
            store_chunk<DT>(static_cast<T *>(a.res_out) + i * a.ld_res_out - off + p, pack<DT>(h[k]), lo, hi);
        if (p < end) {
            y_of(k, p, y);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = 0.f;
        }
        if constexpr (!Q) {
            store_chunk<DT>(static_cast<T *>(a.out) + i * a.ld_out - off + p, pack<DT>(y), lo, hi);
        } else {
            if (a.quant > 0) {                         // (rows start at a chunk)
#pragma unroll
                for (int e = 0; e < V; ++e)
                    if (p + e >= end) y[e] = 0.f;
                uint32_t m = magnitude_max(0u, y);
                for (int o = 1; o < a.quant / V; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                scale = group_scale(m);
                by = Divisor(scale);
                if (p < end && p % a.quant == 0) a.scales[i * a.groups + p / a.quant] = scale;
            }
            if (p >= end) continue;
            store_e4m3<V>(static_cast<uint8_t *>(a.out) + i * a.ld_out - off + p, y, by, off - p,
                          static_cast<int>(end - p));
        }
    }
}

// The gradient with any strides and lengths: dx by a CTA per row, in two passes.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) mbt_layernorm_dx_rows_kernel(const LayerNormGradArgs a) {
    using T = typename Elem<DT>::type;
    __shared__ float red[2 * kRowThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t i = blockIdx.x; i < a.M; i += gridDim.x) {
        const T *dy = static_cast<const T *>(a.dy) + i * a.ld_dy;
        const T *h = static_cast<const T *>(a.h) + i * a.ld_h;
        const T *dr = a.dres ? static_cast<const T *>(a.dres) + i * a.ld_dres : nullptr;
        T *dx = static_cast<T *>(a.dx) + i * a.ld_dx;
        const float mean = a.mean[i], rstd = a.rstd[i];
        float level = 0.f, along = 0.f;
        uint32_t none = 0;
        for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads) {
            const float g = Elem<DT>::widen(dy[j]) * weight_at(a.w, a.wdt, a.woff, j);
            level += g;
            along += g * ((Elem<DT>::widen(h[j]) - mean) * rstd);
        }
        block_reduce<kRowThreads>(level, none, red);
        block_reduce<kRowThreads>(along, none, red);
        level /= static_cast<float>(a.N);
        along /= static_cast<float>(a.N);
        for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads) {
            const float g = Elem<DT>::widen(dy[j]) * weight_at(a.w, a.wdt, a.woff, j);
            const float xh = (Elem<DT>::widen(h[j]) - mean) * rstd;
            const float d = rstd * (g - level - xh * along);
            dx[j] = Elem<DT>::round(d + (dr ? Elem<DT>::widen(dr[j]) : 0.f));
        }
    }
}

// Partial sums of dw and db: CTA (b, s) takes 128 columns of the rows of split s.
template <int DT>
__global__ void __launch_bounds__(kColThreads) mbt_layernorm_dw_rows_kernel(const LayerNormGradArgs a) {
    using T = typename Elem<DT>::type;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x;
    if (j >= a.N) return;
    const int64_t s = blockIdx.y, lo = s * a.M / a.splits, hi = (s + 1) * a.M / a.splits;
    float sw = 0.f, sb = 0.f;
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        float w[4] = {}, b[4] = {};
        const int n = static_cast<int>(min(hi - i0, int64_t{32}));
        auto add = [&](int k, int64_t i) {
            const float dy = Elem<DT>::widen(static_cast<const T *>(a.dy)[i * a.ld_dy + j]);
            w[k] += dy * ((Elem<DT>::widen(static_cast<const T *>(a.h)[i * a.ld_h + j]) - a.mean[i]) * a.rstd[i]);
            b[k] += dy;
        };
        int i = 0;
        for (; i + 4 <= n; i += 4)
#pragma unroll
            for (int k = 0; k < 4; ++k) add(k, i0 + i + k);
        for (; i < n; ++i) add(0, i0 + i);
        sw += pair_sum(w);
        sb += pair_sum(b);
    }
    a.partial[s * a.N + j] = sw;
    a.partial[(a.splits + s) * a.N + j] = sb;
}

// dw (blockIdx.y 0) and db (1) from their partial sums: 32 columns a CTA, 16 threads a
// column, each adding every 16th split, four sums side by side, then the threads' in pairs.
__global__ void __launch_bounds__(32 * kFinishRows) mbt_layernorm_finish_kernel(const LayerNormGradArgs a) {
    __shared__ float part[kFinishRows][32];
    const int l = threadIdx.x & 31, s0 = threadIdx.x >> 5;
    const int64_t j = blockIdx.x * 32ll + l;
    float *out = blockIdx.y ? a.db : a.dw;
    if (!out) return;
    const float *from = a.partial + blockIdx.y * a.splits * a.N;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float sum[4] = {};
    if (j < a.N) {
#pragma unroll 10
        for (int64_t s = s0; s < a.splits; s += kFinishRows) {
            const float v = sum[0] + from[s * a.N + j];
            sum[0] = sum[1], sum[1] = sum[2], sum[2] = sum[3], sum[3] = v;
        }
    }
    part[s0][l] = pair_sum(sum);
    __syncthreads();
    if (s0 != 0 || j >= a.N) return;
    float all[kFinishRows];
#pragma unroll
    for (int s = 0; s < kFinishRows; ++s) all[s] = part[s][l];
    out[j] = pair_sum(all);
}

template <int DT, int C>
cudaError_t launch_ln_forward(const LayerNormVecArgs &va, dim3 grid, int threads, cudaStream_t s) {
    const bool q = va.a.quant != MBT_QUANT_NONE;
    if (va.a.res)
        return q ? launch_grid(mbt_layernorm_kernel<DT, C, true, true>, grid, threads, s, va)
                 : launch_grid(mbt_layernorm_kernel<DT, C, true, false>, grid, threads, s, va);
    return q ? launch_grid(mbt_layernorm_kernel<DT, C, false, true>, grid, threads, s, va)
             : launch_grid(mbt_layernorm_kernel<DT, C, false, false>, grid, threads, s, va);
}

template <int DT>
cudaError_t ln_forward_any(const LayerNormArgs &a, cudaStream_t s) {
    constexpr int V = Elem<DT>::kVec, es = 16 / V;
    const int ph = phase_of(a.x, a.ld_x, es);
    bool same = ph >= 0 && a.N > 0;
    if (a.res) same = same && phase_of(a.res, a.ld_res, es) == ph;
    if (a.res_out) same = same && phase_of(a.res_out, a.ld_res_out, es) == ph;
    if (a.quant == MBT_QUANT_NONE) same = same && phase_of(a.out, a.ld_out, es) == ph;
    if (a.quant > 0) same = same && ph == 0;           // a group is whole lanes' chunks
    if (a.M == 1 && ph >= 0 && !same)                  // (no pitch then)
        same = phase_of(a.x, 0, es) == 0 && (!a.res || phase_of(a.res, 0, es) == 0) &&
               (!a.res_out || phase_of(a.res_out, 0, es) == 0) &&
               (a.quant != MBT_QUANT_NONE || phase_of(a.out, 0, es) == 0) && a.N > 0;
    int sms = 0, optin = 0;
    if (device_limits(&sms, &optin) != MBT_OK) return cudaErrorUnknown;
    LayerNormVecArgs va{a, 0, 0, 0, a.M > 1 && ph > 0};
    const int64_t chunks = (a.N + (va.phased ? V - 1 : 0) + V - 1) / V;
    if (!same || chunks > 4 * 1024) {
        const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.M, 1 << 20)));
        return launch_grid(mbt_layernorm_rows_kernel<DT>, grid, kRowThreads, s, a);
    }
    // as in the root-mean-square norm
    int tpr = a.quant > 0 ? 32 : 8;
    while (tpr < 1024 && (tpr * 2 < chunks || (tpr < chunks && a.M * tpr * 2 <= 1024ll * sms))) tpr *= 2;
    va.tpr = tpr;
    va.wmode = weight_mode(a.w, a.wdt, DT);
    va.bmode = weight_mode(a.b, a.wdt, DT);
    const int threads = tpr > 32 ? tpr : 128, rows = threads / tpr;
    if ((a.M + rows - 1) / rows > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>((a.M + rows - 1) / rows));
    const int64_t c = (chunks + tpr - 1) / tpr;
    return c <= 1   ? launch_ln_forward<DT, 1>(va, grid, threads, s)
           : c <= 2 ? launch_ln_forward<DT, 2>(va, grid, threads, s)
                    : launch_ln_forward<DT, 4>(va, grid, threads, s);
}

// Any strides and lengths: column sums of dw and db in splits of rows, then dx, which may
// overwrite dy.
template <int DT>
int ln_backward_any(LayerNormGradArgs a, cudaStream_t s) {
    int sms = 0, smem = 0;
    int rc = device_limits(&sms, &smem);
    if (rc != MBT_OK) return rc;
    const int64_t cols = (a.N + kColThreads - 1) / kColThreads;
    if (a.dw || a.db) {
        // enough CTAs of 128 columns to fill the device, at least 32 rows each
        a.splits = std::max<int64_t>(1, std::min<int64_t>((a.M + 31) / 32, 16 * sms / cols));
        a.splits = std::min<int64_t>(a.splits, 65535);
        WorkspaceHold hold;
        void *scratch = nullptr;
        rc = hold.scratch(s, static_cast<size_t>(a.splits) * a.N * 8, &scratch);
        if (rc != MBT_OK) return rc;
        a.partial = static_cast<float *>(scratch);
        const dim3 grid(static_cast<unsigned>(cols), static_cast<unsigned>(a.splits));
        cudaError_t e = launch_grid(mbt_layernorm_dw_rows_kernel<DT>, grid, kColThreads, s, a);
        if (e == cudaSuccess)
            e = launch_grid(mbt_layernorm_finish_kernel, dim3(static_cast<unsigned>((a.N + 31) / 32), 2), 32 * kFinishRows, s, a);
        if (e != cudaSuccess) return MBT_ERR_CUDA;
    }
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.M, 1 << 20)));
    return launch_grid(mbt_layernorm_dx_rows_kernel<DT>, grid, kRowThreads, s, a) == cudaSuccess ? MBT_OK
                                                                                                : MBT_ERR_CUDA;
}

}  // namespace

template <int DT>
cudaError_t layernorm_forward(const LayerNormArgs &a, cudaStream_t s) { return ln_forward_any<DT>(a, s); }
template <int DT>
int layernorm_backward(const LayerNormGradArgs &a, cudaStream_t s) { return ln_backward_any<DT>(a, s); }

}  // namespace mbt
