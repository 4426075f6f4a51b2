// Kernels of tile_layernorm and tile_layernorm_backward, for one element type per
// translation unit (mbtile_layernorm_f16.cu, _bf16.cu, _f32.cu).  They share the norm's
// parts: rows in 16-byte chunks by address, rows in registers, the ring of rows in shared
// memory, the plan of a ring (mbtile_norm.cuh).
//
// The variance is summed from deviations, in a second pass over the row's elements
// where they are held: sums of squares would lose the variance of rows whose mean is
// large against it (fp32, mean 1000, deviation 1: the third digit).  The deviations are from
// the rounded sum's mean, which is some units in the last place off; of rows that vary by less
// than that it would be seen in y (fp32, 16384 times 12345.678, eps 1e-5: 0.9 instead of 0).  So
// their own mean, the shift, is summed in the same pass and taken into account:
//   m = sum h / N   s = sum (h - m) / N   mean = m + s   var = sum (h - m)^2 / N - s^2
#pragma once

#include "mbtile_norm.cuh"

namespace mbt {
namespace {

// The statistics of a row.  m, s, q: means of the elements, of the deviations from m and of
// their squares.  A shift that is not finite (rows with an infinity, or whose sum is one) is
// left out: the mean stays m then, and what the deviations make NaN is NaN without it.
__device__ __forceinline__ float row_shift(float s) { return fabsf(s) < __uint_as_float(0x7f800000u) ? s : 0.f; }
__device__ __forceinline__ float row_variance(float s, float q) {
    const float v = fmaf(-s, s, q);
    return v < 0.f ? 0.f : v;                          // (NaN stays NaN)
}

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
        const float n = static_cast<float>(a.N), mean = a.N ? sum / n : 0.f;
        float ss = 0.f;
        sum = 0.f;
        for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads) {
            const float d = h_at(j) - mean;
            sum += d;
            ss += d * d;
        }
        block_reduce<kRowThreads>(sum, amax, red);
        block_reduce<kRowThreads>(ss, amax, red);
        const float shift = row_shift(a.N ? sum / n : 0.f);
        const float rstd = 1.f / sqrtf((a.N ? row_variance(shift, ss / n) : 0.f) + a.eps);
        auto y_of = [&](float h, int64_t j) {
            return (h - mean - shift) * rstd * weight_at(a.w, a.wdt, a.woff, j) + (a.b ? load_any(a.b, a.wdt, j) : 0.f);
        };
        if (threadIdx.x == 0) {
            a.mean[i] = mean + shift;
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

// `tpr` threads hold a row in registers, C chunks each: one pass over memory.  For calls of few
// rows, whose time is a launch and a row's latency with two or three sums in turn (one row of
// 4096 to e4m3 3.6 us, 600 x 2048 3.65), and 16-bit rows of more than 16384 elements whose weight
// or bias is of another type, not aligned or with an offset, which the ring does not take (bf16
// 2000 x 32001 with a residual and fp32 weights 269 us; with bf16 ones by the ring 153).
template <int DT, int C, bool RES, bool Q>
__global__ void __launch_bounds__(1024) mbt_layernorm_kernel(const __grid_constant__ LayerNormVecArgs va) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    __shared__ float red[3][32];
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
    float w0[C > 1 ? 1 : V], b0[C > 1 ? 1 : V];        // one chunk a thread: its weights beside it, on their way at once
    {
        uint4 xv[C], rv[RES ? C : 1];
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int64_t p = static_cast<int64_t>(t + k * tpr) * V;
            xv[k] = make_uint4(0, 0, 0, 0);
            if (RES) rv[k] = make_uint4(0, 0, 0, 0);
            if constexpr (C == 1)
#pragma unroll
                for (int e = 0; e < V; ++e) w0[e] = b0[e] = 0.f;
            if (p >= end) continue;
            const int lo = p < off ? off : 0, hi = end - p < V ? static_cast<int>(end - p) : V;
            xv[k] = load_chunk<DT>(x + p, lo, hi);
            if (RES) rv[k] = load_chunk<DT>(r + p, lo, hi);
            if constexpr (C == 1) {
                load_weight<DT>(a.w, va.wmode, a.wdt, a.woff, p, off, a.N, w0);
                load_bias<DT>(a.b, va.bmode, a.wdt, p, off, a.N, b0);
            }
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
    // the sum over the row, in all of its threads; and two of them, in whole warps the first by
    // the lower lanes and the second by the upper ones
    auto row_sum = [&](float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < tpr) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (tpr > 32) {                                // one row per CTA
            if ((t & 31) == 0) red[0][t >> 5] = v;
            __syncthreads();
            v = warp_sum((t & 31) < (tpr >> 5) ? red[0][t & 31] : 0.f);
        }
        return v;
    };
    auto row_sums = [&](float &v, float &u) {
        if (tpr < 32) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                if (o < tpr) {
                    v += __shfl_xor_sync(0xffffffffu, v, o);
                    u += __shfl_xor_sync(0xffffffffu, u, o);
                }
            return;
        }
        const int lane = t & 31, l = t & 15, warps = tpr >> 5;
        float f = (lane & 16 ? u : v) + __shfl_xor_sync(0xffffffffu, lane & 16 ? v : u, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
        if (tpr > 32) {
            float *const to = red[1 + (lane >> 4)];
            if (l == 0) to[t >> 5] = f;
            __syncthreads();
            f = (l < warps ? to[l] : 0.f) + (l + 16 < warps ? to[l + 16] : 0.f);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o);
        }
        v = __shfl_sync(0xffffffffu, f, 0);
        u = __shfl_sync(0xffffffffu, f, 16);
    };
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) sum += h[k][e];
    const float n = static_cast<float>(a.N), mean = row_sum(sum) / n;
    float ss = 0.f;
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int64_t p = static_cast<int64_t>(t + k * tpr) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float d = h[k][e] - mean;
            if (p + e >= off && p + e < end) sum += d, ss += d * d;
        }
    }
    row_sums(sum, ss);
    const float shift = row_shift(sum / n);
    const float rstd = 1.f / sqrtf(row_variance(shift, ss / n) + a.eps), lead = -shift * rstd;
    auto y_of = [&](int k, int64_t p, float (&y)[V]) {
        float b[V];
        if constexpr (C > 1) {
            load_weight<DT>(a.w, va.wmode, a.wdt, a.woff, p, off, a.N, y);
            load_bias<DT>(a.b, va.bmode, a.wdt, p, off, a.N, b);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = w0[e], b[e] = b0[e];
        }
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = fmaf(h[k][e] - mean, rstd, lead) * y[e] + b[e];
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
        a.mean[i] = mean + shift;
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

// Rows too long for the ring, all of whose chunks are whole but the last: a CTA holds dy and h
// of a row in registers, C chunks a thread: dx in one pass over memory.  C = 0: rows too long
// for that, too, are read twice (the second time from the caches).
template <int DT, int C, bool RES>
__global__ void __launch_bounds__(1024) mbt_layernorm_dx_kernel(const __grid_constant__ LayerNormGradArgs a,
                                                                const int wmode) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    __shared__ float red[2][32];
    const int tpr = blockDim.x, t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int64_t i = blockIdx.x;
    const T *dy = static_cast<const T *>(a.dy) + i * a.ld_dy, *h = static_cast<const T *>(a.h) + i * a.ld_h;
    const T *dr = static_cast<const T *>(a.dres) + (RES ? i * a.ld_dres : 0);
    T *dx = static_cast<T *>(a.dx) + i * a.ld_dx;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float mean = a.mean[i], rstd = a.rstd[i];
    const int count = C ? C : static_cast<int>((a.N + static_cast<int64_t>(tpr) * V - 1) / (static_cast<int64_t>(tpr) * V));
    auto part = [&](int64_t p) { return a.N - p < V ? static_cast<int>(a.N - p) : V; };   // elements of a chunk
    uint4 vy[C ? C : 1], vh[C ? C : 1];
    auto load = [&](int64_t p, uint4 &y, uint4 &x) {
        y = load_chunk<DT>(dy + p, 0, part(p));
        x = load_chunk<DT>(h + p, 0, part(p));
    };
    if constexpr (C > 0)
#pragma unroll
        for (int k = 0; k < C; ++k) {
            const int64_t p = static_cast<int64_t>(t + k * tpr) * V;
            if (p < a.N) load(p, vy[k], vh[k]);
        }
    float level = 0.f, along = 0.f;
#pragma unroll
    for (int k = 0; k < count; ++k) {
        const int64_t p = static_cast<int64_t>(t + k * tpr) * V;
        if (p >= a.N) continue;
        float y[V], x[V], w[V];
        if constexpr (C == 0) load(p, vy[0], vh[0]);
        unpack<DT>(vy[C ? k : 0], y);
        unpack<DT>(vh[C ? k : 0], x);
        load_weight<DT>(a.w, wmode, a.wdt, a.woff, p, 0, a.N, w);
#pragma unroll
        for (int e = 0; e < V; ++e) {                  // (dy is 0 past the row)
            const float g = y[e] * w[e];
            level += g;
            along += g * ((x[e] - mean) * rstd);
        }
    }
    level = warp_sum(level);
    along = warp_sum(along);
    if (lane == 0) red[0][warp] = level, red[1][warp] = along;
    __syncthreads();
    level = warp_sum(lane < (tpr >> 5) ? red[0][lane] : 0.f) / static_cast<float>(a.N);
    along = warp_sum(lane < (tpr >> 5) ? red[1][lane] : 0.f) / static_cast<float>(a.N);
#pragma unroll
    for (int k = 0; k < count; ++k) {
        const int64_t p = static_cast<int64_t>(t + k * tpr) * V;
        if (p >= a.N) continue;
        float y[V], x[V], w[V], f[V];
        if constexpr (RES) unpack<DT>(load_chunk<DT>(dr + p, 0, part(p)), f);
        if constexpr (C == 0) load(p, vy[0], vh[0]);
        unpack<DT>(vy[C ? k : 0], y);
        unpack<DT>(vh[C ? k : 0], x);
        load_weight<DT>(a.w, wmode, a.wdt, a.woff, p, 0, a.N, w);
#pragma unroll
        for (int e = 0; e < V; ++e)
            y[e] = rstd * (y[e] * w[e] - level - (x[e] - mean) * rstd * along) + (RES ? f[e] : 0.f);
        store_chunk<DT>(dx + p, pack<DT>(y), 0, part(p));
    }
}

// Such rows' partial sums of dw and db: CTA (b, s) takes 128 chunks of columns of the rows of
// split s, a chunk a thread.
template <int DT>
__global__ void __launch_bounds__(kColThreads) mbt_layernorm_dw_kernel(const LayerNormGradArgs a) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t j = (static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x) * V;
    if (j >= a.N) return;
    const int n = a.N - j < V ? static_cast<int>(a.N - j) : V;
    const int64_t s = blockIdx.y, lo = s * a.M / a.splits, hi = (s + 1) * a.M / a.splits;
    float w[V] = {}, b[V] = {};
    for (int64_t i0 = lo; i0 < hi; i0 += 4) {
        uint4 vy[4], vh[4];
        float mean[4], rstd[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            vy[k] = vh[k] = make_uint4(0, 0, 0, 0);
            mean[k] = rstd[k] = 0.f;
            const int64_t i = i0 + k;
            if (i >= hi) continue;
            vy[k] = load_chunk<DT>(static_cast<const T *>(a.dy) + i * a.ld_dy + j, 0, n);
            vh[k] = load_chunk<DT>(static_cast<const T *>(a.h) + i * a.ld_h + j, 0, n);
            mean[k] = a.mean[i], rstd[k] = a.rstd[i];
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float tw = 0.f, tb = 0.f;                  // of four rows: a term goes through a quarter of the additions
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float y[V], x[V];
                unpack<DT>(vy[k], y);
                unpack<DT>(vh[k], x);
                tw += y[e] * ((x[e] - mean[k]) * rstd[k]);
                tb += y[e];
            }
            w[e] += tw;
            b[e] += tb;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (e >= n) break;
        a.partial[s * a.N + j + e] = w[e];
        a.partial[(a.splits + s) * a.N + j + e] = b[e];
    }
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

cudaError_t launch_ln_finish(const LayerNormGradArgs &a, cudaStream_t s) {
    return launch_grid(mbt_layernorm_finish_kernel, dim3(static_cast<unsigned>((a.N + 31) / 32), 2), 32 * kFinishRows, s, a);
}

// ---------------------------------------------------------------------------
// Rows through the ring in shared memory
// ---------------------------------------------------------------------------
// As in mbtile_norm.cuh, with a bias beside the weight, or gradients of both, in each
// thread's registers.  What they do not hold is read where it is used: weights of another
// type than 16-bit rows' from global memory (FLY); rows of more than five chunks a thread
// (the gradient's second pass: of more than two, fp32 four) from their stage once more.

// Sums of a and b over a row's tpr threads, in all of them; red and turn as in row_reduce.
// Of a whole warp's values, the lower lanes add up a and the upper ones b.
__device__ __forceinline__ void row_reduce_two(float &a, float &b, int tpr, float *red, int turn) {
    const int lane = threadIdx.x & 31;
    if (tpr < 32) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            if (o >= tpr) continue;
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        return;
    }
    const bool upper = (lane & 16) != 0;
    float v = (upper ? b : a) + __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, warps = tpr >> 5, first = warp & ~(warps - 1);
        float *s = red + turn * 64 + (upper ? 32 : 0);
        if ((lane & 15) == 0) s[warp] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + first / warps), "r"(tpr) : "memory");
        v = (lane & 15) < warps ? s[first + (lane & 15)] : 0.f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    a = __shfl_sync(0xffffffffu, v, 0);
    b = __shfl_sync(0xffffffffu, v, 16);
}

// A thread's weights or biases (`none` where there are none), C chunks of them, 0 past
// the row: packed in x's type, or read each time (FLY, which an offset to 16-bit weights asks
// for too: weight and offset do not fit their type together).
template <int DT, int C, bool PART, bool FLY>
struct RowVector {
    static constexpr int V = Elem<DT>::kVec;
    static constexpr bool kAgain = DT != MBT_F32 && C * V > 16;   // too many to keep unpacked
    uint4 raw[FLY ? 1 : C];
    const void *from;
    int64_t N;
    int mode, type, t, tpr, off;
    float none, add;
    __device__ __forceinline__ void fetch(int c, float offset, float (&v)[V]) const {
        const int64_t p = static_cast<int64_t>(t + c * tpr) * V;
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = p < N + off ? none : 0.f;
        if (from && p < N + off) load_weight<DT>(from, mode, type, offset, p, off, N, v);
    }
    __device__ __forceinline__ RowVector(const void *src, int how, int wdt, float absent, float offset, int thread,
                                         int threads, int lead, int64_t columns)
        : from(src), N(columns), mode(how), type(wdt), t(thread), tpr(threads), off(lead), none(absent),
          add(src ? offset : 0.f) {
        if constexpr (!FLY)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (!PART && from && add == 0.f) {
                    const int p = (t + c * tpr) * V;
                    raw[c] = make_uint4(0, 0, 0, 0);
                    if (p < N) raw[c] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const typename Elem<DT>::type *>(from) + p));
                } else {
                    float v[V];
                    fetch(c, add, v);
                    raw[c] = pack<DT>(v);
                }
            }
    }
    __device__ __forceinline__ void get(int c, uint32_t zero, float (&v)[V]) const {
        if constexpr (FLY) {
            fetch(c, add, v);
        } else {
            unpack<DT>(kAgain ? again(raw[c], zero) : raw[c], v);
        }
    }
};

// Rows that end inside chunks.  The first and the last chunk of a row may hold other rows'
// elements; what that takes is done by the warps that have those chunks (`edge`, the same in
// a warp) in blocks of their own: the row's other warps wait for them at its sums, and
// branches between a thread's loads keep these from being under way together (bf16 8192 x 8191
// with a residual 232 us with calls for each, 212 in the loops over chunks, 189).
struct EdgeMasks {
    uint4 from[9];           // [k]: all bits of a chunk's elements from k on
};
template <int DT>
__device__ __forceinline__ void edge_masks(EdgeMasks &m) {
    constexpr int V = Elem<DT>::kVec, es = 16 / V;
    if (threadIdx.x > V) return;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int bytes = static_cast<int>(threadIdx.x) * es - 4 * k;   // of this word, to be left out
        w[k] = bytes <= 0 ? ~0u : bytes >= 4 ? 0u : ~0u << (8 * bytes);
    }
    m.from[threadIdx.x] = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void sts128(uint32_t at, const uint4 &v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
// v's elements from one on (a) and below another (b).
__device__ __forceinline__ uint4 between(const uint4 &v, const uint4 &a, const uint4 &b) {
    return make_uint4(v.x & a.x & ~b.x, v.y & a.y & ~b.y, v.z & a.z & ~b.z, v.w & a.w & ~b.w);
}
template <int DT, int C, bool PART>
struct EdgeThread : RingThread<DT, C, PART> {
    using Base = RingThread<DT, C, PART>;
    using T = typename Elem<DT>::type;
    static constexpr int V = Elem<DT>::kVec;
    int last;                // the row's last chunk is some thread's of this number
    int most;                // chunks of a thread of this warp, at most
    bool edge;
    uint32_t masks;
    int64_t tail_row;        // from here on a row's last chunk may not have been copied
    __device__ __forceinline__ EdgeThread(const RingArgs &r, int64_t M, int64_t N, uint32_t ring, const EdgeMasks &m)
        : Base(r, M, N, ring) {
        last = PART ? ((Base::end + V - 1) / V - 1) / r.tpr : 0;
        most = __reduce_max_sync(0xffffffffu, Base::count);
        edge = PART && __any_sync(0xffffffffu, Base::head || Base::tail);
        masks = smem_u32(&m);
        tail_row = min(r.tail[0], r.tail[1]);
        if (r.inputs > 2) tail_row = min(tail_row, r.tail[2]);
        if (r.inputs < 2) tail_row = r.tail[0];
    }
    // No thread of this warp has a chunk c.  Rows may fill little more than half of a class's
    // chunks; asked of the last ones, as each branch costs full rows a little (us, from the third /
    // fourth chunk on / never: bf16 with a residual 8192 x 10000 140 / 138 / 144, 8192 x 16384 165
    // / 162 / 161, gradient 8192 x 10000 155 / 160 / 166, 16384 x 8192 187 / 189 / 188).
    template <int FROM>
    __device__ __forceinline__ bool none(int c) const { return c >= FROM && c >= most; }
    __device__ __forceinline__ bool at_edge(int c) const { return PART && edge && (c == 0 || c == last); }
    // Before a row is read from its stage: other rows' elements in its first and last chunk
    // of the first INPUTS matrices to 0, by the threads that alone read them; and the matrix's
    // own last chunk, which is not copied, from the matrix.
    template <int INPUTS>
    __device__ __forceinline__ void prepare(const RingArgs &r, uint32_t stage, int64_t row) const {
        if (!PART || !edge || !(Base::head || Base::tail) || Base::count == 0) return;
        const int c = Base::count - 1;
        if (row >= tail_row && Base::tail) complete(r, stage, row);
        uint4 v[INPUTS], u[INPUTS];
        const uint32_t at = Base::addr + stage * Base::stage_bytes, to = at + static_cast<uint32_t>(c) * Base::chunk_step;
#pragma unroll
        for (int m = 0; m < INPUTS; ++m) {
            v[m] = lds128(at + m * Base::input_step);
            u[m] = lds128(to + m * Base::input_step);
        }
        const uint4 a = lds128(masks + 16 * Base::lo(0)), b = lds128(masks + 16 * Base::hi(0));
        const uint4 e = lds128(masks + 16 * Base::lo(c)), f = lds128(masks + 16 * Base::hi(c));
#pragma unroll
        for (int m = 0; m < INPUTS; ++m) {
            sts128(at + m * Base::input_step, between(v[m], a, b));
            sts128(to + m * Base::input_step, between(u[m], e, f));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (the stage is copied to again)
    }
    // Others' elements of chunk c to x.
    __device__ __forceinline__ void fill(int c, float x, float (&v)[V]) const {
        if (!at_edge(c)) return;
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < Base::lo(c) || e >= Base::hi(c)) v[e] = x;
    }
    __device__ __forceinline__ void complete(const RingArgs &r, uint32_t stage, int64_t row) const {
        for (int m = 0; m < r.inputs; ++m) {
            if (row < r.tail[m]) continue;
            const int c = Base::count - 1;
            const T *from = reinterpret_cast<const T *>(r.in[m] + row * r.ld[m]) - Base::off + (Base::t + c * r.tpr) * V;
            const uint32_t to = Base::addr + stage * Base::stage_bytes + static_cast<uint32_t>(m) * Base::input_step +
                                static_cast<uint32_t>(c) * Base::chunk_step;
#pragma unroll 1
            for (int e = Base::lo(c); e < Base::hi(c); ++e) {
                if constexpr (V == 8)
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + 2 * e), "h"(*reinterpret_cast<const uint16_t *>(from + e))
                                 : "memory");
                else
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + 4 * e), "f"(from[e]) : "memory");
            }
        }
    }
    // Chunk c of a row, if it is the row's alone; and after all of them the parts of those that
    // are not.
    __device__ __forceinline__ void put_whole(T *to, int c, const float (&v)[V]) const {
        if (!PART || (c < Base::count && Base::whole(c))) *reinterpret_cast<uint4 *>(to) = pack<DT>(v);
    }
    __device__ __forceinline__ void put_part(T *to, int c, const float (&v)[V]) const {
        if (!at_edge(c) || c >= Base::count || Base::whole(c)) return;
        const uint4 p = pack<DT>(v);
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
        const int lo = Base::lo(c), hi = Base::hi(c);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (e < lo || e >= hi) continue;
            if constexpr (V == 8)
                reinterpret_cast<uint16_t *>(to)[e] = static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1)));
            else
                reinterpret_cast<uint32_t *>(to)[e] = w[e];
        }
    }
    __device__ __forceinline__ void put(T *to, int c, const float (&v)[V]) const {
        put_whole(to, c, v);
        put_part(to, c, v);
    }
};

struct LayerNormRing {
    RingArgs r;
    int32_t bmode;           // the bias's access (the weight's: r.wmode)
};

// The gradient.  bf16 16384 x 8192 with a residual 187 us, 5.7 TB/s: 31 instructions an element
// on 62 % of the issue slots; fp32 2047 x 5001 35.6 us, by the latency of a row's turn.
template <int DT, int C, bool RES, bool PART, bool FLY>
__global__ void __launch_bounds__(kRingThreads, 1)
    mbt_layernorm_backward_kernel(const __grid_constant__ LayerNormGradArgs a, const __grid_constant__ LayerNormRing l) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    constexpr bool HOLD = C * V <= 16;                       // deviations and gradients in registers from pass to pass
    const RingArgs &r = l.r;
    extern __shared__ __align__(128) unsigned char dyn_smem[];
    __shared__ __align__(8) RingShared sh;
    __shared__ EdgeMasks masks;
    if constexpr (PART) edge_masks<DT>(masks);
    ring_init(sh, r);
    RingState q(r, smem_u32(dyn_smem), smem_u32(&sh.bars[0]), WaitCtl{kDefaultWaitBudgetNs, &sh.abort_flag, r.status});
    q.start(r, a.M);
    const EdgeThread<DT, C, PART> th(r, a.M, a.N, q.ring, masks);
    const RowVector<DT, C, PART, FLY> wt(a.w, r.wmode, a.wdt, 1.f, a.woff, th.t, r.tpr, th.off, a.N);
    float dw[C][V], db[C][V];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[c][e] = db[c][e] = 0.f;
    const float inv_n = 1.f / static_cast<float>(a.N);
    const int64_t rows = static_cast<int64_t>(gridDim.x) * r.rows;   // from one row of a slot to the next
    T *dx = static_cast<T *>(a.dx) + th.first * a.ld_dx - th.off + th.t * V;
    const int chunk = r.tpr * V;
    int turn = 0;
    float next_mean = 0.f, next_rstd = 0.f;
    if (th.first < a.M) next_mean = __ldg(a.mean + th.first), next_rstd = __ldg(a.rstd + th.first);
    const int turns = row_turns(a.M, th.first - th.k % r.unit_rows, rows);
    const int mine = row_turns(a.M, th.first, rows);
    for (int n = 0; n < turns; ++n, dx += rows * a.ld_dx) {
        const uint32_t z1 = r.zero & n, z2 = r.zero & ~n;
        const float mean = n < mine ? next_mean : 0.f, rstd = n < mine ? next_rstd : 0.f;
        const int64_t i = th.first + n * rows;
        if (n + 1 < mine) next_mean = __ldg(a.mean + i + rows), next_rstd = __ldg(a.rstd + i + rows);
        q.wait();
        const int have = n < mine && q.alive ? th.count : 0;
        if (have) th.template prepare<2>(r, q.stage, i);
        // chunk c of dy and h, 0 where it is not the row's
        auto take = [&](int c, uint4 &vy, uint4 &vh) {
            vy = vh = make_uint4(0, 0, 0, 0);
            if (c >= have) return;
            vy = th.chunk(q.stage, 0, c);
            vh = th.chunk(q.stage, 1, c);
        };
        float xs[HOLD ? C : 1][V], gs[HOLD ? C : 1][V];
        float level = 0.f, along = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (th.template none<2>(c)) continue;
            float dy[V], h[V], w[V];
            uint4 vy, vh;
            take(c, vy, vh);
            unpack<DT>(vy, dy);
            unpack<DT>(vh, h);
            wt.get(c, z1, w);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float xh = (h[e] - mean) * rstd, g = dy[e] * w[e];
                level += g;
                along += g * xh;
                dw[c][e] += dy[e] * xh;
                db[c][e] += dy[e];
                if (HOLD) xs[c][e] = xh, gs[c][e] = g;
            }
        }
        row_reduce_two(level, along, r.tpr, sh.red[0], turn);
        turn ^= 1;
        level *= inv_n;
        along *= inv_n;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (c >= have) continue;
            uint4 vr = make_uint4(0, 0, 0, 0);
            if constexpr (RES) vr = th.chunk(q.stage, 2, c);
            float d[V], f[V];
            if constexpr (RES) unpack<DT>(vr, f);
            if constexpr (HOLD) {
#pragma unroll
                for (int e = 0; e < V; ++e) d[e] = rstd * (gs[c][e] - level - xs[c][e] * along) + (RES ? f[e] : 0.f);
            } else {
                float dy[V], h[V], w[V];
                uint4 vy, vh;
                take(c, vy, vh);
                unpack<DT>(vy, dy);
                unpack<DT>(vh, h);
                wt.get(c, z2, w);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    d[e] = rstd * (dy[e] * w[e] - level - (h[e] - mean) * rstd * along) + (RES ? f[e] : 0.f);
            }
            th.put(dx + c * chunk, c, d);
        }
        q.release(r, a.M);
    }
    q.drain(r.stages);
    if (!a.dw && !a.db) return;
    // every stage has been read: its memory takes the row slots' sums, dw's and then db's
    float *slots = reinterpret_cast<float *>(dyn_smem);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        asm volatile("bar.sync 15, %0;" ::"n"(kRingThreads) : "memory");
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const int j = (th.t + c * r.tpr) * V + e - th.off;
                if (j >= 0 && j < a.N) slots[th.k * a.N + j] = which ? db[c][e] : dw[c][e];
            }
        asm volatile("bar.sync 15, %0;" ::"n"(kRingThreads) : "memory");
        for (int j = threadIdx.x; j < a.N; j += kRingThreads) {
            float sum = slots[j];
            if (r.rows < 8) {
                for (int s = 1; s < r.rows; ++s) sum += slots[s * a.N + j];
            } else {
                float eight[8] = {};
                for (int s = 0; s < r.rows; s += 8)
#pragma unroll
                    for (int k = 0; k < 8; ++k) eight[k] += slots[(s + k) * a.N + j];
                sum = pair_sum(eight);
            }
            a.partial[(static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * a.N + j] = sum;
        }
    }
}

// The norm.  bf16 8192 x 16384 with a residual 163 us, 6.6 TB/s: memory.  6881 x 19504 195 us,
// 5.5 TB/s: 32 instructions an element on 55 % of the issue slots.
template <int DT, int C, bool RES, bool Q, bool PART, bool FLY>
__global__ void __launch_bounds__(kRingThreads, 1)
    mbt_layernorm_ring_kernel(const __grid_constant__ LayerNormArgs a, const __grid_constant__ LayerNormRing l) {
    using T = typename Elem<DT>::type;
    using O = typename std::conditional<Q, uint8_t, T>::type;
    constexpr int V = Elem<DT>::kVec;
    const RingArgs &r = l.r;
    extern __shared__ __align__(128) unsigned char dyn_smem[];
    __shared__ __align__(8) RingShared sh;
    __shared__ EdgeMasks masks;
    if constexpr (PART) edge_masks<DT>(masks);
    ring_init(sh, r);
    RingState q(r, smem_u32(dyn_smem), smem_u32(&sh.bars[0]), WaitCtl{kDefaultWaitBudgetNs, &sh.abort_flag, r.status});
    q.start(r, a.M);
    const EdgeThread<DT, C, PART> th(r, a.M, a.N, q.ring, masks);
    const RowVector<DT, C, PART, FLY> wt(a.w, r.wmode, a.wdt, 1.f, a.woff, th.t, r.tpr, th.off, a.N);
    const RowVector<DT, C, PART, FLY> bt(a.b, l.bmode, a.wdt, 0.f, 0.f, th.t, r.tpr, th.off, a.N);
    const float inv_n = 1.f / static_cast<float>(a.N);
    const int64_t rows = static_cast<int64_t>(gridDim.x) * r.rows;   // from one row of a slot to the next
    const int64_t out_step = rows * a.ld_out, res_step = rows * a.ld_res_out;
    O *out = static_cast<O *>(a.out) + th.first * a.ld_out - th.off + th.t * V;
    T *res = static_cast<T *>(a.res_out) + th.first * a.ld_res_out - th.off + th.t * V;
    const bool write_res = RES && a.res_out != nullptr;
    const int chunk = r.tpr * V;
    int turn = 0;
    const int turns = row_turns(a.M, th.first - th.k % r.unit_rows, rows);
    const int mine = row_turns(a.M, th.first, rows);
    for (int n = 0; n < turns; ++n, out += out_step, res += res_step) {
        const uint32_t z1 = r.zero & n, z2 = r.zero & ~n;
        q.wait();
        const int have = n < mine && q.alive ? th.count : 0;
        const int64_t i = th.first + n * rows;
        if (have) th.template prepare<RES ? 2 : 1>(r, q.stage, i);
        if constexpr (C > 5) {
            // Long rows stay in their stage and are read in each pass, which leaves registers for
            // the weights (read from L2 by every row those take as long as the rest: bf16 6881 x
            // 19504 with a residual 564 us).
            // chunk c of h, 0 where it is not the row's
            auto row = [&](int c, float (&f)[V]) {
                uint4 vx = make_uint4(0, 0, 0, 0), vr = vx;
                if (c < have) {
                    vx = th.chunk(q.stage, 0, c);
                    if constexpr (RES) vr = th.chunk(q.stage, 1, c);
                }
                unpack<DT>(vx, f);
                if constexpr (RES) {
                    float g[V];
                    unpack<DT>(vr, g);
#pragma unroll
                    for (int e = 0; e < V; ++e) f[e] += g[e];
                }
            };
            float sum = 0.f, ss = 0.f;
            uint32_t amax = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (th.template none<3>(c)) continue;
                float f[V];
                row(c, f);
#pragma unroll
                for (int e = 0; e < V; ++e) sum += f[e];
            }
            row_reduce<false>(sum, amax, r.tpr, sh.red[0], turn);
            turn ^= 1;
            const float mean = __fdiv_rn(sum, static_cast<float>(a.N));
            sum = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (c >= have) continue;
                float f[V];
                row(c, f);
                if (write_res) th.put(res + c * chunk, c, f);
                th.fill(c, mean, f);
                const Pair from(-mean);
                Pair part(0.f), dev(0.f);
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const Pair d = Pair(f[e], f[e + 1]) + from;
                    dev = dev + d;
                    part = fma2(d, d, part);
                }
                sum += dev.get().x + dev.get().y;
                ss += part.get().x + part.get().y;
            }
            row_reduce_two(sum, ss, r.tpr, sh.red[0], turn);
            turn ^= 1;
            const float shift = row_shift(sum * inv_n);
            const float rstd = rsqrtf(row_variance(shift, ss * inv_n) + a.eps);
            if (th.t == 0 && n < mine) {
                a.mean[i] = mean + shift;
                a.rstd[i] = rstd;
            }
            auto y_of = [&](int c, uint32_t z, float (&f)[V]) {
                float w[V], b[V];
                row(c, f);
                wt.get(c, z, w);
                bt.get(c, z, b);
                const Pair rr(rstd), lead(-shift * rstd);
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const float2 y = fma2(fma2(Pair(f[e] - mean, f[e + 1] - mean), rr, lead), Pair(w[e], w[e + 1]), Pair(b[e], b[e + 1])).get();
                    f[e] = y.x, f[e + 1] = y.y;
                }
                if (Q) th.fill(c, 0.f, f);
            };
            float scale = 0.f;
            Divisor by;
            if (Q && a.quant == 0) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if (c >= have) continue;
                    float f[V];
                    y_of(c, z1, f);
                    amax = magnitude_max(amax, f);
                }
                float none = 0.f;
                row_reduce<true>(none, amax, r.tpr, sh.red[0], turn);
                turn ^= 1;
                scale = group_scale(amax);
                by = Divisor(scale);
                if (th.t == 0 && n < mine) a.scales[i] = scale;
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (th.template none<3>(c)) continue;
                float f[V];
                y_of(c, z2, f);
                if constexpr (!Q) {
                    if (c < have) th.put(out + c * chunk, c, f);
                } else {
                    if (a.quant > 0) {       // (rows start at a chunk)
                        uint32_t m = c < have ? magnitude_max(0u, f) : 0u;
#pragma unroll
                        for (int o = 1; o < 128 / V; o <<= 1) {
                            if (o >= a.quant / V) break;
                            m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                        }
                        scale = group_scale(m);
                        by = Divisor(scale);
                        const int p = th.t * V + c * chunk;
                        if (c < have && p % a.quant == 0) a.scales[i * a.groups + p / a.quant] = scale;
                    }
                    if (c < have) store_e4m3<V>(out + c * chunk, f, by, th.lo(c), th.hi(c));
                }
            }
            q.release(r, a.M);
            continue;
        }
        float h[C][V];
        {
            uint4 vx[C], vr[RES ? C : 1];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                vx[c] = make_uint4(0, 0, 0, 0);
                if constexpr (RES) vr[c] = make_uint4(0, 0, 0, 0);
                if (c >= have) continue;
                vx[c] = th.chunk(q.stage, 0, c);
                if constexpr (RES) vr[c] = th.chunk(q.stage, 1, c);
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (th.template none<3>(c)) continue;
                unpack<DT>(vx[c], h[c]);
                if constexpr (RES) {
                    float f[V];
                    unpack<DT>(vr[c], f);
#pragma unroll
                    for (int e = 0; e < V; ++e) h[c][e] += f[e];
                }
            }
        }
        q.release(r, a.M);   // the row is in registers now
        float sum = 0.f, ss = 0.f;
        uint32_t amax = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (th.template none<3>(c)) continue;
#pragma unroll
            for (int e = 0; e < V; ++e) sum += h[c][e];
        }
        row_reduce<false>(sum, amax, r.tpr, sh.red[0], turn);
        turn ^= 1;
        const float mean = __fdiv_rn(sum, static_cast<float>(a.N));
        sum = 0.f;
        if constexpr (PART) {
            if (write_res && have) {
#pragma unroll
                for (int c = 0; c < C; ++c) th.put_whole(res + c * chunk, c, h[c]);
                if (th.edge)
#pragma unroll
                    for (int c = 0; c < C; ++c) th.put_part(res + c * chunk, c, h[c]);
            }
            if (th.edge)
#pragma unroll
                for (int c = 0; c < C; ++c) th.fill(c, mean, h[c]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (th.template none<3>(c)) continue;
            if (!PART && c < have && write_res) th.put(res + c * chunk, c, h[c]);
            const Pair from(-mean);
            Pair part(0.f), dev(0.f);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const Pair d = Pair(h[c][e], h[c][e + 1]) + from;   // from here on the deviation
                h[c][e] = d.get().x, h[c][e + 1] = d.get().y;
                dev = dev + d;
                part = fma2(d, d, part);
            }
            if (c < have) sum += dev.get().x + dev.get().y, ss += part.get().x + part.get().y;
        }
        row_reduce_two(sum, ss, r.tpr, sh.red[0], turn);
        turn ^= 1;
        const float shift = row_shift(sum * inv_n);
        const float rstd = rsqrtf(row_variance(shift, ss * inv_n) + a.eps);
        if (th.t == 0 && n < mine) {
            a.mean[i] = mean + shift;
            a.rstd[i] = rstd;
        }
        uint32_t gmax[C];                    // largest magnitude of each chunk's group
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if constexpr (Q) gmax[c] = 0u;
            if (th.template none<3>(c)) continue;
            float w[V], b[V];
            wt.get(c, z1, w);
            bt.get(c, z2, b);
            const Pair rr(rstd), lead(-shift * rstd);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const float2 y = fma2(fma2(Pair(h[c][e], h[c][e + 1]), rr, lead), Pair(w[e], w[e + 1]), Pair(b[e], b[e + 1])).get();
                h[c][e] = y.x, h[c][e + 1] = y.y;
            }
            if constexpr (!Q) {
                if (c < have) th.put_whole(reinterpret_cast<T *>(out + c * chunk), c, h[c]);
            } else {
                th.fill(c, 0.f, h[c]);
                gmax[c] = c < have ? magnitude_max(0u, h[c]) : 0u;
            }
        }
        if (!Q && PART && th.edge && have)
#pragma unroll
            for (int c = 0; c < C; ++c) th.put_part(reinterpret_cast<T *>(out + c * chunk), c, h[c]);
        if constexpr (Q) {
            float scale = 0.f;
            Divisor by;
            if (a.quant == 0) {
#pragma unroll
                for (int c = 0; c < C; ++c) amax = max(amax, gmax[c]);
                float none = 0.f;
                row_reduce<true>(none, amax, r.tpr, sh.red[0], turn);
                turn ^= 1;
                scale = group_scale(amax);
                by = Divisor(scale);
                if (th.t == 0 && n < mine) a.scales[i] = scale;
            } else {                         // (rows start at a chunk)
#pragma unroll
                for (int o = 1; o < 128 / V; o <<= 1) {
                    if (o >= a.quant / V) break;
#pragma unroll
                    for (int c = 0; c < C; ++c) gmax[c] = max(gmax[c], __shfl_xor_sync(0xffffffffu, gmax[c], o));
                }
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (c >= have) continue;
                if (a.quant > 0) {
                    scale = group_scale(gmax[c]);
                    by = Divisor(scale);
                    const int p = th.t * V + c * chunk;
                    if (p % a.quant == 0) a.scales[i * a.groups + p / a.quant] = scale;
                }
                store_e4m3<V>(out + c * chunk, h[c], by, th.lo(c), th.hi(c));
            }
        }
    }
    q.drain(r.stages);
}

template <class K, class A>
cudaError_t launch_ln_ring(K kernel, const RingPlan &p, int bmode, cudaStream_t s, const A &a) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    return launch_pipeline(kernel, p.grid, kRingThreads, p.smem, s, a, LayerNormRing{p.r, bmode});
}

template <int DT, int C, bool PART, bool FLY>
cudaError_t launch_ln_ring_forward(const RingPlan &p, int bmode, const LayerNormArgs &a, cudaStream_t s) {
    const bool q = a.quant != MBT_QUANT_NONE;
    if (a.res)
        return q ? launch_ln_ring(mbt_layernorm_ring_kernel<DT, C, true, true, PART, FLY>, p, bmode, s, a)
                 : launch_ln_ring(mbt_layernorm_ring_kernel<DT, C, true, false, PART, FLY>, p, bmode, s, a);
    return q ? launch_ln_ring(mbt_layernorm_ring_kernel<DT, C, false, true, PART, FLY>, p, bmode, s, a)
             : launch_ln_ring(mbt_layernorm_ring_kernel<DT, C, false, false, PART, FLY>, p, bmode, s, a);
}

template <int DT, int C, bool PART, bool FLY>
cudaError_t launch_ln_ring_backward(const RingPlan &p, const LayerNormGradArgs &a, cudaStream_t s) {
    return a.dres ? launch_ln_ring(mbt_layernorm_backward_kernel<DT, C, true, PART, FLY>, p, 0, s, a)
                  : launch_ln_ring(mbt_layernorm_backward_kernel<DT, C, false, PART, FLY>, p, 0, s, a);
}

// A vector that whole chunks of the rows' type can be read from, or none.
bool plain_vector(int mode) { return mode == kSameWeight || mode == kNoWeight; }

template <int DT>
cudaError_t ln_ring_forward(const RingPlan &p, int bmode, const LayerNormArgs &a, cudaStream_t s) {
    const int c = p.chunks;
    const bool part = p.part || !plain_vector(p.r.wmode) || !plain_vector(bmode);
    if constexpr (DT == MBT_F32) {
        if (c > 5)
            return part ? launch_ln_ring_forward<DT, 8, true, false>(p, bmode, a, s)
                        : launch_ln_ring_forward<DT, 8, false, false>(p, bmode, a, s);
        if (part)
            return c <= 4 ? launch_ln_ring_forward<DT, 4, true, false>(p, bmode, a, s)
                          : launch_ln_ring_forward<DT, 5, true, false>(p, bmode, a, s);
        return c <= 2   ? launch_ln_ring_forward<DT, 2, false, false>(p, bmode, a, s)
               : c <= 4 ? launch_ln_ring_forward<DT, 4, false, false>(p, bmode, a, s)
                        : launch_ln_ring_forward<DT, 5, false, false>(p, bmode, a, s);
    } else {
        if (c > 4)
            return part ? launch_ln_ring_forward<DT, 8, true, false>(p, bmode, a, s)
                        : launch_ln_ring_forward<DT, 8, false, false>(p, bmode, a, s);
        if (a.w && (a.wdt != DT || a.woff != 0.f)) return launch_ln_ring_forward<DT, 4, true, true>(p, bmode, a, s);
        if (part)
            return c <= 2 ? launch_ln_ring_forward<DT, 2, true, false>(p, bmode, a, s)
                          : launch_ln_ring_forward<DT, 4, true, false>(p, bmode, a, s);
        return c <= 1   ? launch_ln_ring_forward<DT, 1, false, false>(p, bmode, a, s)
               : c <= 2 ? launch_ln_ring_forward<DT, 2, false, false>(p, bmode, a, s)
                        : launch_ln_ring_forward<DT, 4, false, false>(p, bmode, a, s);
    }
}

template <int DT>
cudaError_t ln_ring_backward(const RingPlan &p, const LayerNormGradArgs &a, cudaStream_t s) {
    const int c = p.chunks;
    const bool part = p.part || !plain_vector(p.r.wmode);
    if constexpr (DT == MBT_F32) {
        if (part)
            return c <= 4 ? launch_ln_ring_backward<DT, 4, true, false>(p, a, s)
                          : launch_ln_ring_backward<DT, 5, true, false>(p, a, s);
        return c <= 2   ? launch_ln_ring_backward<DT, 2, false, false>(p, a, s)
               : c <= 4 ? launch_ln_ring_backward<DT, 4, false, false>(p, a, s)
                        : launch_ln_ring_backward<DT, 5, false, false>(p, a, s);
    } else {
        if (a.w && (a.wdt != DT || a.woff != 0.f)) return launch_ln_ring_backward<DT, 4, true, true>(p, a, s);
        if (part)
            return c <= 2 ? launch_ln_ring_backward<DT, 2, true, false>(p, a, s)
                          : launch_ln_ring_backward<DT, 4, true, false>(p, a, s);
        return c <= 1   ? launch_ln_ring_backward<DT, 1, false, false>(p, a, s)
               : c <= 2 ? launch_ln_ring_backward<DT, 2, false, false>(p, a, s)
                        : launch_ln_ring_backward<DT, 4, false, false>(p, a, s);
    }
}

// The ring's plan: up to four chunks a thread of 16-bit rows, of fp32 rows up to five; up to
// eight of rows too long for that, forward, where 16-bit rows ask for weights of their type.
// A single stage will do for the longest: forward the next row is copied while this one's is
// stored, and for the gradient (fp32 2000 x 10240 with a residual 71 us) the alternative reads
// rows twice (132; of longer fp32 rows by eight chunks, whose weights it would read each time,
// 2000 x 12000 142 us, without the ring 119).  Rows side by side hide each other's reductions, so few threads take a row
// (us, four chunks / two, forward 8192 x 8192 bf16 with a residual 87 / 121; gradient 16384 x 8192
// 187 / 215, 65536 x 1024 95 / 118; fp32 2047 x 5001, five / four 37 / 52), but for a gradient of
// few turns, where the last one's length and the more instructions of rows that registers do not
// hold count (3001 x 4001 48 / 38, 1024 x 4096 20.4 / 17.5, 8192 x 4096 of 13 turns 61 / 64, 9001
// x 1032 of 7 36 / 39).  Forward eight chunks of 16-bit rows are ahead of four, given the turns:
// with a residual 8192 x 10000 113 / 139, 8192 x 8200 108 / 137, 16384 x 1400 of 7 turns 35 / 39,
// 8192 x 8192 83 / 83, 700 x 8200 of 2 15.9 / 15.6; of parts of chunks 8192 x 8191 160 / 189, 8192
// x 5001 of 13 70 / 80, 4000 x 5001 of 7 to e4m3 84 / 68.  (Forward figures here and at
// ln_ring_pays precede the shift, which cost up to 3 %.)
bool ln_ring_plan(const void *const *in, const int64_t *ld, int inputs, int64_t M, int64_t N, int es, int ph, int min_tpr,
                  int sms, bool gradient, bool plain, RingPlan *p) {
    if (es == 4)
        return ring_plan(in, ld, inputs, M, N, es, ph, 5, min_tpr, sms, p, 5, 1) ||
               (!gradient && ring_plan(in, ld, inputs, M, N, es, ph, 8, min_tpr, sms, p, 0, 1));
    const bool eight = plain && !gradient;
    if (eight && ring_plan(in, ld, inputs, M, N, es, ph, 8, min_tpr, sms, p, 8) &&
        M >= (p->part ? 10ll : 6ll) * p->grid * p->r.rows)
        return true;
    if (!ring_plan(in, ld, inputs, M, N, es, ph, 4, min_tpr, sms, p, 4))
        return eight && ring_plan(in, ld, inputs, M, N, es, ph, 8, min_tpr, sms, p, 8, 1);
    if (!gradient || M >= 6ll * p->grid * p->r.rows) return true;
    return ring_plan(in, ld, inputs, M, N, es, ph, 4, min_tpr, sms, p, 2);
}

// The gradient through the ring; *done says whether it applied.
template <int DT>
int ln_backward_by_ring(LayerNormGradArgs a, cudaStream_t s, int sms, bool *done) {
    constexpr int V = Elem<DT>::kVec, es = 16 / V;
    const int ph = phase_of(a.h, a.ld_h, es);
    bool same = ph >= 0 && phase_of(a.dy, a.ld_dy, es) == ph && phase_of(a.dx, a.ld_dx, es) == ph;
    if (a.dres) same = same && phase_of(a.dres, a.ld_dres, es) == ph;
    const void *in[3] = {a.dy, a.h, a.dres};
    const int64_t ld[3] = {a.ld_dy, a.ld_h, a.ld_dres};
    RingPlan p;
    *done = same && ln_ring_plan(in, ld, a.dres ? 3 : 2, a.M, a.N, es, ph, 8, sms, true, false, &p);
    if (!*done) return MBT_OK;
    int rc = device_status_word(&p.r.status);
    if (rc != MBT_OK) return rc;
    p.r.wmode = weight_mode(a.w, a.wdt, DT);
    a.splits = p.grid;
    WorkspaceHold hold;
    if (a.dw || a.db) {
        void *scratch = nullptr;
        rc = hold.scratch(s, static_cast<size_t>(a.splits) * a.N * 8, &scratch);
        if (rc != MBT_OK) return rc;
        a.partial = static_cast<float *>(scratch);
    }
    cudaError_t e = ln_ring_backward<DT>(p, a, s);
    if (e == cudaSuccess && (a.dw || a.db)) e = launch_ln_finish(a, s);
    return e == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
}

// Where the ring is faster than a row in registers (us, ring / registers): its start is paid
// once a call, so with enough rows, of whatever length: bf16 with a residual 131072 x 512 96
// / 113, 8192 x 8192 85 / 128, 512 x 8192 10.2 / 12.5, 256 x 8192 7.1 / 7.0, 2000 x 512 6.6 /
// 4.4, 6881 x 19504 199 / 390, 152 x 32768 12.2 / 14.4; without, 131072 x 256 31 / 48, 65537 x
// 1001 110 / 141, 304 x 8192 by groups of 128 to e4m3 7.0 / 7.7, 1000 x 1001 8.9 / 4.0.
bool ln_ring_pays(const LayerNormArgs &a, int64_t es) { return a.M * a.N * es >= (5ll << 20); }

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
    const void *in[2] = {a.x, a.res};
    const int64_t ld[2] = {a.ld_x, a.ld_res};
    const bool plain = plain_vector(weight_mode(a.w, a.wdt, DT)) && plain_vector(weight_mode(a.b, a.wdt, DT)) && a.woff == 0.f;
    RingPlan p;
    if (same && ln_ring_pays(a, es) &&
        ln_ring_plan(in, ld, a.res ? 2 : 1, a.M, a.N, es, ph, a.quant > 0 ? 32 : 8, sms, false, plain, &p)) {
        if (device_status_word(&p.r.status) != MBT_OK) return cudaErrorUnknown;
        p.r.wmode = weight_mode(a.w, a.wdt, DT);
        return ln_ring_forward<DT>(p, weight_mode(a.b, a.wdt, DT), a, s);
    }
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

template <int DT, int C>
cudaError_t launch_ln_dx(const LayerNormGradArgs &a, int wmode, int threads, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.M));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.dres ? cudaLaunchKernelEx(&cfg, mbt_layernorm_dx_kernel<DT, C, true>, a, wmode)
                  : cudaLaunchKernelEx(&cfg, mbt_layernorm_dx_kernel<DT, C, false>, a, wmode);
}

// Any strides and lengths: column sums of dw and db in splits of rows, then dx, which may
// overwrite dy.  Rows that begin at whole chunks by chunks, with dx's in registers (bf16 1000 x
// 24000 with a residual 178 us by elements).
template <int DT>
int ln_backward_any(LayerNormGradArgs a, cudaStream_t s) {
    constexpr int V = Elem<DT>::kVec, es = 16 / V;
    int sms = 0, smem = 0;
    int rc = device_limits(&sms, &smem);
    if (rc != MBT_OK) return rc;
    bool done = false;
    rc = ln_backward_by_ring<DT>(a, s, sms, &done);
    if (rc != MBT_OK || done) return rc;
    const bool read = phase_of(a.dy, a.ld_dy, es) == 0 && phase_of(a.h, a.ld_h, es) == 0;
    const int64_t chunks = (a.N + V - 1) / V;
    if (a.dw || a.db) {
        // enough CTAs of 128 columns (or chunks) to fill the device, at least 32 rows each
        const int64_t cols = ((read ? chunks : a.N) + kColThreads - 1) / kColThreads;
        a.splits = std::max<int64_t>(1, std::min<int64_t>((a.M + 31) / 32, 16 * sms / cols));
        a.splits = std::min<int64_t>(a.splits, 65535);
        WorkspaceHold hold;
        void *scratch = nullptr;
        rc = hold.scratch(s, static_cast<size_t>(a.splits) * a.N * 8, &scratch);
        if (rc != MBT_OK) return rc;
        a.partial = static_cast<float *>(scratch);
        const dim3 grid(static_cast<unsigned>(cols), static_cast<unsigned>(a.splits));
        cudaError_t e = read ? launch_grid(mbt_layernorm_dw_kernel<DT>, grid, kColThreads, s, a)
                             : launch_grid(mbt_layernorm_dw_rows_kernel<DT>, grid, kColThreads, s, a);
        if (e == cudaSuccess) e = launch_ln_finish(a, s);
        if (e != cudaSuccess) return MBT_ERR_CUDA;
    }
    if (read && phase_of(a.dx, a.ld_dx, es) == 0 && (!a.dres || phase_of(a.dres, a.ld_dres, es) == 0) &&
        a.M <= 0x7fffffff) {
        const int wmode = weight_mode(a.w, a.wdt, DT);
        const int threads = static_cast<int>(std::min<int64_t>(1024, (chunks + 31) / 32 * 32));
        const int64_t c = (chunks + threads - 1) / threads;
        const cudaError_t e = c <= 1   ? launch_ln_dx<DT, 1>(a, wmode, threads, s)
                              : c <= 2 ? launch_ln_dx<DT, 2>(a, wmode, threads, s)
                              : c <= 4 ? launch_ln_dx<DT, 4>(a, wmode, threads, s)
                                       : launch_ln_dx<DT, 0>(a, wmode, threads, s);
        return e == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
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
