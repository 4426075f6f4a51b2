// tile_rmsnorm and tile_rmsnorm_backward: the root-mean-square norm over a
// matrix's rows, with the residual's addition, and its gradient.
//
//   h = x + r    rstd_i = (mean_j h_ij^2 + eps)^(-1/2)    y = h rstd (w + o)
//   xh = h rstd  g = dy (w + o)  c_i = mean_j(g xh)
//   dx = rstd (g - xh c) + dres          dw_j = sum_i dy xh
//
// Both read and write every matrix once and compute a handful of operations
// per element: device memory bounds them.  All sums are fp32.
#include <algorithm>

#include "mbtile_elem.cuh"
#include "mbtile_layer.h"
#include "mbtile_ptx.cuh"

namespace mbt {
namespace {

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

constexpr int kRowThreads = 512;

// Sum and largest magnitude over the CTA, the same in every thread.
template <int THREADS>
__device__ __forceinline__ void block_reduce(float &sum, uint32_t &amax, float *red) {
    sum = warp_sum(sum);
    amax = __reduce_max_sync(0xffffffffu, amax);
    uint32_t *redm = reinterpret_cast<uint32_t *>(red + THREADS / 32);
    __syncthreads();   // the last round's reads of red are over
    if ((threadIdx.x & 31) == 0) {
        red[threadIdx.x >> 5] = sum;
        redm[threadIdx.x >> 5] = amax;
    }
    __syncthreads();
    sum = 0.f;
    amax = 0;
#pragma unroll
    for (int k = 0; k < THREADS / 32; ++k) {
        sum += red[k];
        amax = max(amax, redm[k]);
    }
}

__device__ __forceinline__ float weight_at(const void *w, int wdt, float woff, int64_t j) {
    return w ? load_any(w, wdt, j) + woff : 1.f;
}

// Any strides and lengths: a CTA per row, two passes over it (the second one's
// reads hit the caches), one element per access.
template <int DT>
__global__ void __launch_bounds__(kRowThreads) mbt_rmsnorm_rows_kernel(const NormArgs a) {
    using T = typename Elem<DT>::type;
    __shared__ float red[2 * kRowThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t i = blockIdx.x; i < a.M; i += gridDim.x) {
        const T *x = static_cast<const T *>(a.x) + i * a.ld_x;
        const T *r = a.res ? static_cast<const T *>(a.res) + i * a.ld_res : nullptr;
        T *ro = a.res_out ? static_cast<T *>(a.res_out) + i * a.ld_res_out : nullptr;
        auto h_at = [&](int64_t j) {
            return Elem<DT>::widen(x[j]) + (r ? Elem<DT>::widen(r[j]) : 0.f);
        };
        float ss = 0.f;
        uint32_t amax = 0;
        for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads) {
            const float h = h_at(j);
            ss += h * h;
            if (a.quant == 0) amax = max(amax, magnitude(h * weight_at(a.w, a.wdt, a.woff, j)));
        }
        block_reduce<kRowThreads>(ss, amax, red);
        const float rstd = 1.f / sqrtf((a.N ? ss / static_cast<float>(a.N) : 0.f) + a.eps);
        if (threadIdx.x == 0) a.rstd[i] = rstd;
        if (a.quant <= 0) {
            const float scale = group_scale(magnitude(__uint_as_float(amax) * rstd));
            const float inv = 1.f / scale;
            if (a.quant == 0 && threadIdx.x == 0) a.scales[i] = scale;
            for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads) {
                const float h = h_at(j);
                const float y = h * rstd * weight_at(a.w, a.wdt, a.woff, j);
                if (a.quant == 0)
                    static_cast<uint8_t *>(a.out)[i * a.ld_out + j] =
                        static_cast<uint8_t>(to_e4m3x2(y * inv, 0.f));
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
                    y[k] = h * rstd * weight_at(a.w, a.wdt, a.woff, j);
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
                    static_cast<uint8_t *>(a.out)[i * a.ld_out + j] =
                        static_cast<uint8_t>(to_e4m3x2(y[k] * (1.f / scale), 0.f));
                    if (j % a.quant == 0) a.scales[i * a.groups + j / a.quant] = scale;
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Forward, 16-byte accesses
// ---------------------------------------------------------------------------
// Rows of any length and pitch are cut into 16-byte chunks by address, not from
// their first element: a row that starts `off` elements into a chunk has its
// first and last chunk in part, and everything between is moved 16 bytes at a
// time.  (All matrices of a call must start rows at the same place in a chunk;
// mbt_rmsnorm_rows_kernel takes the others.)

// Elements [lo, hi) of the chunk at p, the others 0; and their store.
template <int DT>
__device__ __noinline__ uint4 load_part(const typename Elem<DT>::type *p, int lo, int hi) {
    using T = typename Elem<DT>::type;
    union {
        uint4 v;
        T e[Elem<DT>::kVec];
    } u;
    u.v = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < Elem<DT>::kVec; ++e)
        if (e >= lo && e < hi) u.e[e] = p[e];
    return u.v;
}

template <int DT>
__device__ __noinline__ void store_part(typename Elem<DT>::type *p, uint4 v, int lo, int hi) {
    using T = typename Elem<DT>::type;
    union {
        uint4 v;
        T e[Elem<DT>::kVec];
    } u;
    u.v = v;
#pragma unroll
    for (int e = 0; e < Elem<DT>::kVec; ++e)
        if (e >= lo && e < hi) p[e] = u.e[e];
}

template <int DT>
__device__ __forceinline__ uint4 load_chunk(const typename Elem<DT>::type *p, int lo, int hi) {
    constexpr int V = Elem<DT>::kVec;
    // (not a read-only load: outputs may be the inputs themselves)
    if (lo <= 0 && hi >= V) return *reinterpret_cast<const uint4 *>(p);
    return load_part<DT>(p, lo, hi);
}

template <int DT>
__device__ __forceinline__ void store_chunk(typename Elem<DT>::type *p, const uint4 &v, int lo, int hi) {
    constexpr int V = Elem<DT>::kVec;
    if (lo <= 0 && hi >= V)
        *reinterpret_cast<uint4 *>(p) = v;
    else
        store_part<DT>(p, v, lo, hi);
}

// How the weight is read: none, as 16-byte vectors of x's type or of fp32, or by
// element (rows that start inside a chunk, other types).
enum { kNoWeight = 0, kSameWeight = 1, kF32Weight = 2, kAnyWeight = 3 };

template <int DT>
__device__ __forceinline__ void load_weight(const void *w, int mode, int wdt, float woff, int64_t j,
                                            int64_t N, float (&f)[Elem<DT>::kVec]) {
    constexpr int V = Elem<DT>::kVec;
    if (mode == kNoWeight) {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = 1.f;
        return;
    }
    if (mode == kSameWeight) {
        unpack<DT>(__ldg(reinterpret_cast<const uint4 *>(static_cast<const typename Elem<DT>::type *>(w) + j)), f);
    } else if (mode == kF32Weight) {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + j + e));
            f[e] = v.x, f[e + 1] = v.y, f[e + 2] = v.z, f[e + 3] = v.w;
        }
    } else {
#pragma unroll 1
        for (int e = 0; e < V; ++e) {
            const float v = j + e >= 0 && j + e < N ? load_any(w, wdt, j + e) : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == e) f[i] = v;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] += woff;
}

struct NormVecArgs {
    NormArgs a;
    int32_t tpr, wmode;      // threads per row (a power of two), weight access
    int32_t phased;          // rows may start inside a chunk
};

// `tpr` threads hold a row in registers, C chunks each: one pass over memory.
// Bound by device memory; rows in flight on an SM (CTAs that fit) hide the
// latency between a row's loads and its stores.
template <int DT, int C, bool RES, bool Q>
__global__ void __launch_bounds__(1024) mbt_rmsnorm_kernel(const __grid_constant__ NormVecArgs va) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    __shared__ float red[32];
    __shared__ uint32_t redm[32];
    const NormArgs &a = va.a;
    const int tpr = va.tpr, t = threadIdx.x & (tpr - 1);
    const int64_t i = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = i < a.M;
    const int off = va.phased ? static_cast<int>((i * a.ld_x) & (V - 1)) : 0;
    const int64_t end = live ? a.N + off : 0;          // in elements from the first chunk
    const T *x = static_cast<const T *>(a.x) + i * a.ld_x - off;
    const T *r = static_cast<const T *>(a.res) + i * a.ld_res - off;
    asm volatile("griddepcontrol.wait;" ::: "memory");
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
    auto h_of = [&](int k, float (&h)[V]) {
        unpack<DT>(xv[k], h);
        if (RES) {
            float f[V];
            unpack<DT>(rv[k], f);
#pragma unroll
            for (int e = 0; e < V; ++e) h[e] += f[e];
        }
    };
    float ss = 0.f;
    uint32_t amax = 0;
#pragma unroll
    for (int k = 0; k < C; ++k) {
        float h[V];
        h_of(k, h);
#pragma unroll
        for (int e = 0; e < V; ++e) ss += h[e] * h[e];
        const int64_t p = static_cast<int64_t>(t + k * tpr) * V;
        if (Q && a.quant == 0 && p < end) {
            float w[V];
            load_weight<DT>(a.w, va.wmode, a.wdt, a.woff, p - off, a.N, w);
#pragma unroll
            for (int e = 0; e < V; ++e) amax = max(amax, magnitude(h[e] * w[e]));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (o >= tpr) continue;
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (Q) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    if (tpr > 32) {                                    // one row per CTA
        if ((t & 31) == 0) {
            red[t >> 5] = ss;
            if (Q) redm[t >> 5] = amax;
        }
        __syncthreads();
        const int warps = tpr >> 5, l = t & 31;
        ss = l < warps ? red[l] : 0.f;
        ss = warp_sum(ss);
        if (Q) amax = __reduce_max_sync(0xffffffffu, l < warps ? redm[l] : 0u);
    }
    const float rstd = 1.f / sqrtf(ss / static_cast<float>(a.N) + a.eps);
    float scale = 0.f, inv = 0.f;
    if (Q && a.quant == 0) {
        scale = group_scale(magnitude(__uint_as_float(amax) * rstd));
        inv = 1.f / scale;
    }
    if (live && t == 0) {
        a.rstd[i] = rstd;
        if (Q && a.quant == 0) a.scales[i] = scale;
    }
#pragma unroll
    for (int k = 0; k < C; ++k) {
        const int64_t p = static_cast<int64_t>(t + k * tpr) * V;
        if (!Q && p >= end) continue;
        const int lo = p < off ? off : 0, hi = end - p < V ? static_cast<int>(end - p) : V;
        float h[V], y[V];
        h_of(k, h);
        if (RES && p < end && a.res_out)
            store_chunk<DT>(static_cast<T *>(a.res_out) + i * a.ld_res_out - off + p, pack<DT>(h), lo, hi);
        if (p < end) {
            load_weight<DT>(a.w, va.wmode, a.wdt, a.woff, p - off, a.N, y);
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] *= h[e] * rstd;
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = 0.f;
        }
        if constexpr (!Q) {
            store_chunk<DT>(static_cast<T *>(a.out) + i * a.ld_out - off + p, pack<DT>(y), lo, hi);
        } else {
            if (a.quant > 0) {                         // (rows start at a chunk)
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < V; ++e) m = max(m, magnitude(y[e]));
                for (int o = 1; o < a.quant / V; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
                scale = group_scale(m);
                inv = 1.f / scale;
                if (p < end && p % a.quant == 0) a.scales[i * a.groups + p / a.quant] = scale;
            }
            if (p >= end) continue;
            uint32_t q[V / 4];
#pragma unroll
            for (int e = 0; e < V; e += 4)
                q[e / 4] = to_e4m3x2(y[e] * inv, y[e + 1] * inv) |
                           to_e4m3x2(y[e + 2] * inv, y[e + 3] * inv) << 16;
            uint8_t *o = static_cast<uint8_t *>(a.out) + i * a.ld_out - off + p;
            if (lo == 0 && hi == V && (reinterpret_cast<uintptr_t>(o) & (V - 1)) == 0) {
                if constexpr (V == 8)
                    *reinterpret_cast<uint2 *>(o) = make_uint2(q[0], q[1]);
                else
                    *reinterpret_cast<uint32_t *>(o) = q[0];
            } else {
#pragma unroll 1
                for (int e = lo; e < hi; ++e) o[e] = static_cast<uint8_t>((V == 8 && e >= 4 ? q[V / 4 - 1] : q[0]) >> (8 * (e & 3)));
            }
        }
    }
}

template <int DT>
__global__ void __launch_bounds__(kRowThreads) mbt_rmsnorm_dx_rows_kernel(const NormGradArgs a) {
    using T = typename Elem<DT>::type;
    __shared__ float red[2 * kRowThreads / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t i = blockIdx.x; i < a.M; i += gridDim.x) {
        const T *dy = static_cast<const T *>(a.dy) + i * a.ld_dy;
        const T *h = static_cast<const T *>(a.h) + i * a.ld_h;
        const T *dr = a.dres ? static_cast<const T *>(a.dres) + i * a.ld_dres : nullptr;
        T *dx = static_cast<T *>(a.dx) + i * a.ld_dx;
        const float rstd = a.rstd[i];
        float dot = 0.f;
        uint32_t none = 0;
        for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads)
            dot += Elem<DT>::widen(dy[j]) * weight_at(a.w, a.wdt, a.woff, j) *
                   (Elem<DT>::widen(h[j]) * rstd);
        block_reduce<kRowThreads>(dot, none, red);
        const float c = dot / static_cast<float>(a.N);
        for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads) {
            const float g = Elem<DT>::widen(dy[j]) * weight_at(a.w, a.wdt, a.woff, j);
            const float d = rstd * (g - Elem<DT>::widen(h[j]) * rstd * c);
            dx[j] = Elem<DT>::round(d + (dr ? Elem<DT>::widen(dr[j]) : 0.f));
        }
    }
}

constexpr int kColThreads = 128;

// dw's partial sums: CTA (b, s) takes 128 columns of the rows of split s.
template <int DT>
__global__ void __launch_bounds__(kColThreads) mbt_rmsnorm_dw_rows_kernel(const NormGradArgs a) {
    using T = typename Elem<DT>::type;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x;
    if (j >= a.N) return;
    const int64_t s = blockIdx.y, lo = s * a.M / a.splits, hi = (s + 1) * a.M / a.splits;
    float sum = 0.f;
#pragma unroll 4
    for (int64_t i = lo; i < hi; ++i)
        sum += Elem<DT>::widen(static_cast<const T *>(a.dy)[i * a.ld_dy + j]) *
               (Elem<DT>::widen(static_cast<const T *>(a.h)[i * a.ld_h + j]) * a.rstd[i]);
    a.partial[s * a.N + j] = sum;
}

// dw from its partial sums, in split order.
__global__ void __launch_bounds__(kColThreads) mbt_rmsnorm_dw_finish_kernel(const NormGradArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t j = static_cast<int64_t>(blockIdx.x) * kColThreads + threadIdx.x;
    if (j >= a.N) return;
    float sum = 0.f;
#pragma unroll 8
    for (int64_t s = 0; s < a.splits; ++s) sum += a.partial[s * a.N + j];
    a.dw[j] = sum;
}

int64_t elem_bytes(int dtype) { return dtype == MBT_F32 ? 4 : 2; }

bool float_type(int dtype) { return dtype == MBT_F16 || dtype == MBT_BF16 || dtype == MBT_F32; }

bool aligned_elem(const void *p, int dtype) {
    return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(elem_bytes(dtype)) == 0;
}

constexpr int64_t kMaxIndex = int64_t{1} << 46;   // elements an address may be away

// Row pitch (0 => N) and its bounds.
bool pitch(int64_t *ld, int64_t M, int64_t N) {
    if (*ld == 0) *ld = N;
    return *ld >= N && (M == 0 || *ld <= kMaxIndex / M);
}

// Where the rows of a matrix start in 16-byte chunks: -1 if not known from the
// first row on, else the pitch's part beyond whole chunks (0: every row at a chunk).
int phase_of(const void *p, int64_t ld, int64_t es) {
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return -1;
    return static_cast<int>(ld * es % 16);
}

int weight_mode(const void *w, int wdt, int dtype, bool phased) {
    if (!w) return kNoWeight;
    if (phased || reinterpret_cast<uintptr_t>(w) % 16 != 0) return kAnyWeight;
    return wdt == dtype ? kSameWeight : wdt == MBT_F32 ? kF32Weight : kAnyWeight;
}

template <int DT, int C>
cudaError_t launch_forward(const NormVecArgs &va, dim3 grid, int threads, cudaStream_t s) {
    const bool q = va.a.quant != MBT_QUANT_NONE;
    if (va.a.res)
        return q ? launch_grid(mbt_rmsnorm_kernel<DT, C, true, true>, grid, threads, s, va)
                 : launch_grid(mbt_rmsnorm_kernel<DT, C, true, false>, grid, threads, s, va);
    return q ? launch_grid(mbt_rmsnorm_kernel<DT, C, false, true>, grid, threads, s, va)
             : launch_grid(mbt_rmsnorm_kernel<DT, C, false, false>, grid, threads, s, va);
}

template <int DT>
cudaError_t forward(const NormArgs &a, cudaStream_t s) {
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
    NormVecArgs va{a, 0, 0, a.M > 1 && ph > 0};
    const int64_t chunks = (a.N + (va.phased ? V - 1 : 0) + V - 1) / V;
    if (!same || chunks > 4 * 1024) {
        const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.M, 1 << 20)));
        return launch_grid(mbt_rmsnorm_rows_kernel<DT>, grid, kRowThreads, s, a);
    }
    // Two chunks a thread while that keeps a row within a CTA; a warp at least
    // where groups of up to 128 columns are reduced, and all of a CTA for a few
    // rows, where the time is one row's latency.
    int tpr = a.quant > 0 ? 32 : 8;
    while (tpr < 1024 && (tpr * 2 < chunks || (a.M < 64 && tpr < chunks))) tpr *= 2;
    va.tpr = tpr;
    va.wmode = weight_mode(a.w, a.wdt, DT, va.phased);
    // (a vector of the weight past its end: only whole chunks read as vectors)
    if (a.N % V != 0 && va.wmode != kNoWeight) va.wmode = kAnyWeight;
    const int threads = tpr > 32 ? tpr : 128, rows = threads / tpr;
    if ((a.M + rows - 1) / rows > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>((a.M + rows - 1) / rows));
    const int64_t c = (chunks + tpr - 1) / tpr;
    return c <= 1   ? launch_forward<DT, 1>(va, grid, threads, s)
           : c <= 2 ? launch_forward<DT, 2>(va, grid, threads, s)
                    : launch_forward<DT, 4>(va, grid, threads, s);
}

}  // namespace
}  // namespace mbt

extern "C" int tile_rmsnorm(const void *x, const void *residual, const void *weight, void *out,
                            void *residual_out, float *scales, float *rstd, int64_t M, int64_t N,
                            int64_t ld_x, int64_t ld_res, int64_t ld_out, int64_t ld_res_out,
                            int dtype, int weight_dtype, int quant, float eps, float weight_offset,
                            void *stream) {
    using namespace mbt;
    if (M < 0 || N < 0 || N > 0x7fffffff || !float_type(dtype) ||
        (weight && !float_type(weight_dtype)) || !(eps >= 0.f))
        return MBT_ERR_ARG;
    if (quant != MBT_QUANT_NONE && quant != MBT_QUANT_ROW && quant != 32 && quant != 64 && quant != 128)
        return MBT_ERR_UNSUPPORTED;
    if (!pitch(&ld_x, M, N) || !pitch(&ld_res, M, N) || !pitch(&ld_out, M, N) ||
        !pitch(&ld_res_out, M, N))
        return MBT_ERR_ARG;
    if (M == 0) return MBT_OK;
    if (!rstd || (N > 0 && (!x || !out)) || (quant != MBT_QUANT_NONE) != (scales != nullptr) ||
        (residual_out && !residual))
        return MBT_ERR_ARG;
    if (!aligned_elem(x, dtype) || !aligned_elem(residual, dtype) ||
        !aligned_elem(residual_out, dtype) || (weight && !aligned_elem(weight, weight_dtype)) ||
        (quant == MBT_QUANT_NONE && !aligned_elem(out, dtype)) || !aligned_elem(rstd, MBT_F32) ||
        !aligned_elem(scales, MBT_F32))
        return MBT_ERR_ALIGN;
    const NormArgs a{x,      residual, weight, out,        residual_out, scales,
                     rstd,   M,        N,      ld_x,       ld_res,       ld_out,
                     ld_res_out, quant > 0 ? (N + quant - 1) / quant : 1,
                     weight_dtype, quant, eps, weight_offset};
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == MBT_F16    ? forward<MBT_F16>(a, s)
                          : dtype == MBT_BF16 ? forward<MBT_BF16>(a, s)
                                              : forward<MBT_F32>(a, s);
    return e == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
}

extern "C" int tile_rmsnorm_backward(const void *dy, const void *h, const float *rstd,
                                     const void *weight, const void *dresidual, void *dx,
                                     float *dweight, int64_t M, int64_t N, int64_t ld_dy,
                                     int64_t ld_h, int64_t ld_dres, int64_t ld_dx, int dtype,
                                     int weight_dtype, float weight_offset, void *stream) {
    using namespace mbt;
    if (M < 0 || N < 0 || N > 0x7fffffff || !float_type(dtype) ||
        (weight && !float_type(weight_dtype)))
        return MBT_ERR_ARG;
    if (!pitch(&ld_dy, M, N) || !pitch(&ld_h, M, N) || !pitch(&ld_dres, M, N) || !pitch(&ld_dx, M, N))
        return MBT_ERR_ARG;
    if (N == 0) return MBT_OK;
    if (M > 0 && (!dy || !h || !rstd || !dx)) return MBT_ERR_ARG;
    if (!aligned_elem(dy, dtype) || !aligned_elem(h, dtype) || !aligned_elem(dresidual, dtype) ||
        !aligned_elem(dx, dtype) || (weight && !aligned_elem(weight, weight_dtype)) ||
        !aligned_elem(rstd, MBT_F32) || !aligned_elem(dweight, MBT_F32))
        return MBT_ERR_ALIGN;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M == 0) {
        if (!dweight) return MBT_OK;
        return cudaMemsetAsync(dweight, 0, static_cast<size_t>(N) * 4, s) == cudaSuccess ? MBT_OK
                                                                                          : MBT_ERR_CUDA;
    }
    int sms = 0, smem = 0;
    int rc = device_limits(&sms, &smem);
    if (rc != MBT_OK) return rc;
    NormGradArgs a{dy, h, weight, dresidual, rstd, dx, dweight, nullptr, M, N, ld_dy, ld_h, ld_dres,
                   ld_dx, 1, weight_dtype, weight_offset};
    const unsigned cols = static_cast<unsigned>((N + kColThreads - 1) / kColThreads);
    cudaError_t e = cudaSuccess;
    if (dweight) {
        // enough CTAs of 128 columns to fill the device, at least 32 rows each
        a.splits = std::max<int64_t>(1, std::min<int64_t>((M + 31) / 32, 16 * sms / cols));
        a.splits = std::min<int64_t>(a.splits, 65535);
        void *scratch = nullptr;
        rc = owned_scratch(stream, static_cast<size_t>(a.splits) * N * 4, &scratch);
        if (rc != MBT_OK) return rc;
        a.partial = static_cast<float *>(scratch);
        const dim3 grid(cols, static_cast<unsigned>(a.splits));
        // before dx, which may overwrite dy or h
        e = dtype == MBT_F16    ? launch_grid(mbt_rmsnorm_dw_rows_kernel<MBT_F16>, grid, kColThreads, s, a)
            : dtype == MBT_BF16 ? launch_grid(mbt_rmsnorm_dw_rows_kernel<MBT_BF16>, grid, kColThreads, s, a)
                                : launch_grid(mbt_rmsnorm_dw_rows_kernel<MBT_F32>, grid, kColThreads, s, a);
        if (e == cudaSuccess) e = launch_grid(mbt_rmsnorm_dw_finish_kernel, dim3(cols), kColThreads, s, a);
        if (e != cudaSuccess) return MBT_ERR_CUDA;
    }
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(M, 1 << 20)));
    e = dtype == MBT_F16    ? launch_grid(mbt_rmsnorm_dx_rows_kernel<MBT_F16>, grid, kRowThreads, s, a)
        : dtype == MBT_BF16 ? launch_grid(mbt_rmsnorm_dx_rows_kernel<MBT_BF16>, grid, kRowThreads, s, a)
                            : launch_grid(mbt_rmsnorm_dx_rows_kernel<MBT_F32>, grid, kRowThreads, s, a);
    return e == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
}
