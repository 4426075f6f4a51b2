// Kernels of tile_rmsnorm and tile_rmsnorm_backward, for one element type per
// translation unit (mbtile_norm_f16.cu, _bf16.cu, _f32.cu).
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "mbtile_elem.cuh"
#include "mbtile_layer.h"
#include "mbtile_ptx.cuh"
#include "mbtile_rows.h"

namespace mbt {
namespace {

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

// The sum of v in pairs.  The last sums of dw are taken like this, several side by
// side and then in pairs, as rounding errors grow with the root of the additions that
// a term goes through (fp32, 16000 x 64: 2.8 u with all in series).
template <int V>
__device__ __forceinline__ float pair_sum(float (&v)[V]) {
#pragma unroll
    for (int n = V / 2; n > 0; n /= 2)
#pragma unroll
        for (int k = 0; k < n; ++k) v[k] += v[k + n];
    return v[0];
}

// Any strides and lengths: a CTA per row, two passes over it (the second one's
// reads hit the caches), one element per access, which bounds it by instructions
// and latency (bf16 1024 x 65536, residual: 402 us, 1.3 TB/s).
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
            if (a.quant == 0 && threadIdx.x == 0) a.scales[i] = scale;
            for (int64_t j = threadIdx.x; j < a.N; j += kRowThreads) {
                const float h = h_at(j);
                const float y = h * rstd * weight_at(a.w, a.wdt, a.woff, j);
                if (a.quant == 0)
                    static_cast<uint8_t *>(a.out)[i * a.ld_out + j] =
                        static_cast<uint8_t>(to_e4m3x2(y / scale, 0.f));
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
                        static_cast<uint8_t>(to_e4m3x2(y[k] / scale, 0.f));
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
// element (other alignments and types).
enum { kNoWeight = 0, kSameWeight = 1, kF32Weight = 2, kAnyWeight = 3 };

// Eight words, moved down by `words` (0..4) and, with `half`, by 16 bits more: the
// first four.  The amounts are the same in a whole warp.
__device__ __forceinline__ uint4 shift_words(uint4 lo, uint4 hi, int words, bool half) {
    uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int s = 4; s > 0; s >>= 1)
        if (words & s)
#pragma unroll
            for (int i = 0; i + s < 8; ++i) v[i] = v[i + s];
    if (half)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __funnelshift_r(v[i], v[i + 1], 16);
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// The weights of the row chunk whose first element is column j = p - off, 0 out of
// range: with off > 0 they lie in two of the weight's own chunks.
template <int DT>
__device__ __forceinline__ void load_weight(const void *w, int mode, int wdt, float woff, int64_t p,
                                            int off, int64_t N, float (&f)[Elem<DT>::kVec]) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    const int64_t j = p - off;
    if (mode == kNoWeight) {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = 1.f;
        return;
    }
    if (mode == kSameWeight) {
        const T *wt = static_cast<const T *>(w);
        auto chunk = [&](int64_t q) {      // the weight's own chunk from element q on
            return q < N ? load_chunk<DT>(wt + q, 0, N - q < V ? static_cast<int>(N - q) : V)
                         : make_uint4(0, 0, 0, 0);
        };
        uint4 v = chunk(p);
        if (off) {
            const uint4 u = p >= V ? chunk(p - V) : make_uint4(0, 0, 0, 0);
            constexpr int es = 16 / V;
            const int bytes = (V - off) * es;
            v = shift_words(u, v, bytes >> 2, (bytes & 2) != 0);
        }
        unpack<DT>(v, f);
    } else if (mode == kF32Weight && off == 0 && p + V <= N) {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(w) + j + e));
            f[e] = v.x, f[e + 1] = v.y, f[e + 2] = v.z, f[e + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e) f[e] = j + e >= 0 && j + e < N ? load_any(w, wdt, j + e) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] += woff;
}

// V values by their scale as e4m3 at o, elements [lo, hi) of them.
template <int V>
__device__ __forceinline__ void store_e4m3(uint8_t *o, const float (&y)[V], const Divisor &by, int lo, int hi) {
    uint32_t q[V / 4];
#pragma unroll
    for (int e = 0; e < V; e += 4) {
        const float2 a = by.minus(y[e], y[e + 1]), b = by.minus(y[e + 2], y[e + 3]);
        q[e / 4] = (to_e4m3x2(a.x, a.y) | to_e4m3x2(b.x, b.y) << 16) ^ 0x80808080u;
    }
    if (lo <= 0 && hi >= V && (reinterpret_cast<uintptr_t>(o) & (V - 1)) == 0) {
        if constexpr (V == 8)
            *reinterpret_cast<uint2 *>(o) = make_uint2(q[0], q[1]);
        else
            *reinterpret_cast<uint32_t *>(o) = q[0];
        return;
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        if (e >= lo && e < hi) o[e] = static_cast<uint8_t>(q[e / 4] >> (8 * (e & 3)));
}

struct NormVecArgs {
    NormArgs a;
    int32_t tpr, wmode;      // threads per row (a power of two), weight access
    int32_t phased;          // rows may start inside a chunk
};

// `tpr` threads hold a row in registers, C chunks each: one pass over memory.
// Bound by device memory; rows in flight on an SM (CTAs that fit) hide the
// latency between a row's loads and its stores (bf16, residual: 131072 x 512
// 80 us, 6.7 TB/s; 256 x 8192 3.6 us, 4.7 TB/s from L2; one row of 8192 to e4m3 3.5
// us, the latency of a launch and a row).  To e4m3 the short rows are bound by
// instructions (131072 x 512 by groups of 128, no residual: 99 us, 2.0 TB/s).
// (Times here and below are of the kernels alone, replayed from graphs.)
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
            load_weight<DT>(a.w, va.wmode, a.wdt, a.woff, p, off, a.N, w);
#pragma unroll
            for (int e = 0; e < V; ++e) w[e] *= h[e];
            amax = magnitude_max(amax, w);
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
    float scale = 0.f;
    Divisor by;
    if (Q && a.quant == 0) {
        scale = group_scale(magnitude(__uint_as_float(amax) * rstd));
        by = Divisor(scale);
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
            load_weight<DT>(a.w, va.wmode, a.wdt, a.woff, p, off, a.N, y);
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

// ---------------------------------------------------------------------------
// Rows through a ring in shared memory
// ---------------------------------------------------------------------------
// A persistent CTA per SM of 16 warps, cut into units: the tpr threads of a row, or
// a warp that holds several short rows.  Each unit keeps its next rows of every
// input matrix on their way into stages of its own by 1-D bulk copies (the row's
// 16-byte-aligned window of bytes, so any pitch will do) and works on the stage that
// has landed, a thread always on the same columns.  That keeps the weight, and the
// gradient of the weight, in registers for the whole kernel, and loads under way
// while rows are reduced and written.  A unit's first warp refills a stage once
// the unit has read it; one ring for the whole CTA made every unit wait for the
// slowest (gradient of bf16 65536 x 128: twice the time; 16384 x 2048 7 % more), and a warp of its own for refilling would be the 17th and cost each
// thread 32 of its 128 registers.  A row costs a thread 200 to 300 instructions
// whatever its length (barrier, shuffles, addresses), so threads take up to 32
// elements each rather than rows fewer threads.  (32 warps of half the registers
// were slower in the forward: bf16 4096 x 4096 by 16 %.)
//
// Long rows are bound by device memory (fp16 16384 x 16384, residual: gradient
// 319 us, 6.7 TB/s; forward 364 us, 5.9 TB/s, 357 to 366 from run to run); calls of a
// few turns by the start, the last turn's latency and that overhead (bf16 4096 x 4096,
// residual: 22.4 us, 6.0 TB/s; gradient 32.1, 4.2; bf16 2047 x 8192 to e4m3 by groups of
// 128: 29.7, 4.0, with 48 % of the issue slots taken; fp32 4097 x 8191 at an odd pitch:
// 63.5, 4.2, its warps waiting for one another at the row's barrier).
constexpr int kRingThreads = 512;
constexpr int kRingStages = 8;
constexpr int kRingBars = kRingThreads / 32 * kRingStages;   // of all units
constexpr int kRingBytes = 208 * 1024;   // shared memory for the stages

struct RingArgs {
    const char *in[3];       // forward: x, residual; backward: dy, h, dresidual
    int64_t ld[3];           // pitches in bytes
    int64_t tail[3];         // first rows whose last chunk is not copied
    int32_t row_bytes;
    int32_t inputs;
    int32_t tpr, rows;       // threads per row, rows at a time
    int32_t unit_threads;    // that share a ring: a row's, or a warp of several rows
    int32_t unit_rows;
    uint32_t stage_bytes;    // of a unit
    int32_t stages;
    int32_t slot;            // bytes of a row's window, at most
    int32_t phased;          // rows may start inside a chunk
    int32_t wmode;
    uint32_t zero;           // 0, not known to the compiler
    int32_t *status;
};

// The unit's first warp: the copies of its rows from `row` on to `to`.
__device__ __forceinline__ void ring_fill(const RingArgs &r, int64_t M, uint32_t to, uint32_t full, int64_t row) {
    const int lane = threadIdx.x & 31;
    const int rows = static_cast<int>(min(M - row, static_cast<int64_t>(r.unit_rows)));
    uint32_t total = 0;
    for (int i = lane; i < rows * r.inputs; i += 32)
        total += row_window(row + i % rows, r.tail[i / rows], r.row_bytes, r.ld[i / rows], r.phased).bytes;
    total = __reduce_add_sync(0xffffffffu, total);
    if (lane == 0) mbar_arrive_expect_tx(full, total);
    __syncwarp();
    for (int i = lane; i < rows * r.inputs; i += 32) {
        const int m = i / rows, k = i - m * rows;
        const RowWindow win = row_window(row + k, r.tail[m], r.row_bytes, r.ld[m], r.phased);
        if (win.bytes > 0)
            bulk_load_1d(to + static_cast<uint32_t>((m * r.unit_rows + k) * r.slot), r.in[m] + win.start,
                         static_cast<uint32_t>(win.bytes), full);
    }
}

// A unit's ring and its position in it, the same in every one of its warps.
struct RingState {
    uint32_t ring, full, empty;   // shared memory: the stages, their barriers
    int64_t row, step;            // the first of the unit's rows to be copied next, from turn to turn
    bool lead;                    // its first warp
    WaitCtl w;
    uint32_t stage = 0, phase = 0;
    bool alive = true;            // no wait of this warp has run out

    __device__ __forceinline__ RingState(const RingArgs &r, uint32_t memory, uint32_t bars, const WaitCtl &wait) : w(wait) {
        const uint32_t unit = threadIdx.x / r.unit_threads;
        ring = memory + unit * r.stages * r.stage_bytes;
        full = bars + 8 * unit * r.stages;
        empty = full + 8 * kRingBars;
        row = static_cast<int64_t>(blockIdx.x) * r.rows + unit * r.unit_rows;
        step = static_cast<int64_t>(gridDim.x) * r.rows;
        lead = threadIdx.x - unit * r.unit_threads < 32;
    }
    // The unit's first rows.
    __device__ __forceinline__ void start(const RingArgs &r, int64_t M) {
        if (!lead) return;
        for (int s = 0; s < r.stages; ++s, row += step)
            if (row < M) ring_fill(r, M, ring + s * r.stage_bytes, full + 8 * s, row);
    }
    // A warp whose wait has run out goes through the rows without work, so that
    // the CTA's barriers are complete.
    __device__ __forceinline__ void wait() {
        if (alive && !__all_sync(0xffffffffu, mbar_try_wait(full + 8 * stage, phase) ||
                                                  wait_bounded(full + 8 * stage, phase, w, true))) {
            report_timeout(w, 1, stage, phase);
            *w.abort = 1;
            alive = false;
        }
    }
    // This warp has read its stage.
    __device__ __forceinline__ void release(const RingArgs &r, int64_t M) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(empty + 8 * stage);
        if (lead && alive && row < M) {
            if (__all_sync(0xffffffffu, wait_bounded(empty + 8 * stage, phase, w, true))) {
                ring_fill(r, M, ring + stage * r.stage_bytes, full + 8 * stage, row);
                row += step;
            } else {
                report_timeout(w, 0, stage, phase);
                *w.abort = 1;
                alive = false;
            }
        }
        if (++stage == static_cast<uint32_t>(r.stages)) stage = 0, phase ^= 1;
    }
    // After a wait that ran out: the copies under way land before the CTA leaves.
    __device__ __forceinline__ void drain(int stages) {
        if (!lead || (threadIdx.x & 31) != 0 || !*w.abort) return;
        for (int s = 0; s < stages; ++s)
            for (uint32_t p = 0; p < 2; ++p) wait_bounded(full + 8 * s, p, w, false);
    }
};

// The sum of v (and the largest amax) over a row's tpr threads, in all of them.
// red: two sets of 32 words for sums and 32 for magnitudes, used in turn, so that
// one barrier per row is enough.
template <bool MAX>
__device__ __forceinline__ void row_reduce(float &v, uint32_t &amax, int tpr, float *red, int turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        if (o >= tpr) continue;
        v += __shfl_xor_sync(0xffffffffu, v, o);
        if (MAX) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    if (tpr <= 32) return;
    const int warp = threadIdx.x >> 5, warps = tpr >> 5, first = warp & ~(warps - 1), lane = threadIdx.x & 31;
    float *s = red + turn * 64;
    uint32_t *m = reinterpret_cast<uint32_t *>(s + 32);
    if (lane == 0) {
        s[warp] = v;
        if (MAX) m[warp] = amax;
    }
    asm volatile("bar.sync %0, %1;" ::"r"(1 + first / warps), "r"(tpr) : "memory");
    v = lane < warps ? s[first + lane] : 0.f;
    v = warp_sum(v);
    if (MAX) amax = __reduce_max_sync(0xffffffffu, lane < warps ? m[first + lane] : 0u);
}

struct RingShared {
    uint64_t bars[2 * kRingBars];    // full, empty: of each unit's stages
    float red[2][64];
    int abort_flag;
};

__device__ __forceinline__ void ring_init(RingShared &sh, const RingArgs &r) {
    for (int i = threadIdx.x; i < r.stages * kRingThreads / r.unit_threads; i += kRingThreads) {
        mbar_init(smem_u32(&sh.bars[i]), 1);
        mbar_init(smem_u32(&sh.bars[kRingBars + i]), r.unit_threads / 32);
    }
    if (threadIdx.x == 0) sh.abort_flag = 0;
    fence_barrier_init();
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// v, in a form that neither compiler nor assembler knows to be v (zero is a kernel
// argument and something of the row), so that it is unpacked where it is used
// instead of its fp32 values (twice the registers) being kept from pass to pass,
// and those of the weight from row to row.
__device__ __forceinline__ uint4 again(const uint4 &v, uint32_t zero) {
    return make_uint4(v.x ^ zero, v.y ^ zero, v.z ^ zero, v.w ^ zero);
}

// A thread's weights, C chunks of them, 0 past the row: packed in x's type, or
// (W32: fp32 weights of 16-bit rows) as fp32.
template <int DT, int C, bool PART, bool W32>
struct RingWeights {
    static constexpr int V = Elem<DT>::kVec;
    float f[W32 ? C : 1][V];
    uint4 raw[W32 ? 1 : C];
    float woff;
    __device__ __forceinline__ void load(const RingArgs &r, const void *w, int wdt, float offset, int t, int off,
                                         int64_t N) {
        woff = offset;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int p = (t + c * r.tpr) * V;
            if constexpr (!PART && !W32) {
                raw[c] = make_uint4(0, 0, 0, 0);
                if (p < N)
                    raw[c] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const typename Elem<DT>::type *>(w) + p));
            } else {
                float v[V];
#pragma unroll
                for (int e = 0; e < V; ++e) v[e] = 0.f;
                if (p < N + off) load_weight<DT>(w, r.wmode, wdt, 0.f, p, off, N, v);
                if constexpr (W32)
#pragma unroll
                    for (int e = 0; e < V; ++e) f[c][e] = v[e];
                else
                    raw[c] = pack<DT>(v);
            }
        }
        if (w == nullptr) woff = 0.f;
    }
    __device__ __forceinline__ void get(int c, uint32_t zero, float (&v)[V]) const {
        if constexpr (W32) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] = f[c][e];
        } else {
            unpack<DT>(again(raw[c], zero), v);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] += woff;
    }
};

// A thread's place in the rows of its slot: the same chunks of every one of them.
// (The host makes the grid such that all rows of a slot start at the same place in
// a chunk.)
template <int DT, int C, bool PART>
struct RingThread {
    static constexpr int V = Elem<DT>::kVec;
    int t, k;                // thread of the row, row slot
    int off, end;            // the row's elements are [off, end) from its first chunk on
    int count;               // chunks of this thread
    bool head, tail;         // its first, its last chunk is not the row's alone
    int64_t first;           // first row
    uint32_t addr, chunk_step, input_step, stage_bytes;   // shared memory

    __device__ __forceinline__ RingThread(const RingArgs &r, int64_t M, int64_t N, uint32_t ring) {
        t = threadIdx.x & (r.tpr - 1);
        k = threadIdx.x / r.tpr;
        first = static_cast<int64_t>(blockIdx.x) * r.rows + k;
        off = PART ? row_window(first < M ? first : 0, M, 0, r.ld[0], r.phased).lead / (16 / V) : 0;
        end = static_cast<int>(N) + off;
        const int chunks = (end + V - 1) / V;
        count = t < chunks ? min(C, (chunks - t + r.tpr - 1) / r.tpr) : 0;
        head = PART && off > 0 && t == 0;
        tail = PART && end % V != 0 && count > 0 && t + (count - 1) * r.tpr == chunks - 1;
        chunk_step = static_cast<uint32_t>(r.tpr) * 16u;
        input_step = static_cast<uint32_t>(r.unit_rows * r.slot);
        stage_bytes = r.stage_bytes;
        addr = ring + static_cast<uint32_t>(k % r.unit_rows * r.slot + t * 16);
    }
    // Chunk c of input m in the stage at `stage`.
    __device__ __forceinline__ uint4 chunk(uint32_t stage, int m, int c) const {
        return lds128(addr + stage * stage_bytes + static_cast<uint32_t>(m) * input_step +
                      static_cast<uint32_t>(c) * chunk_step);
    }
    __device__ __forceinline__ bool whole(int c) const {
        return !PART || !((head && c == 0) || (tail && c == count - 1));
    }
    // Elements of chunk c that are the row's: [lo, hi).
    __device__ __forceinline__ int lo(int c) const { return head && c == 0 ? off : 0; }
    __device__ __forceinline__ int hi(int c) const { return tail && c == count - 1 ? end & (V - 1) : V; }
    // The matrix's partial last chunk is not copied: from the matrix itself.
    __device__ __forceinline__ void last_chunk(const RingArgs &r, int m, int c, int64_t row, uint4 &v) const {
        using T = typename Elem<DT>::type;
        if (row >= r.tail[m] && tail && c == count - 1)
            v = load_part<DT>(reinterpret_cast<const T *>(r.in[m] + row * r.ld[m]) - off + (t + c * r.tpr) * V, lo(c), hi(c));
    }
    // Other rows' elements to 0.
    __device__ __forceinline__ void mask(int c, float (&v)[V]) const {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < lo(c) || e >= hi(c)) v[e] = 0.f;
    }
    __device__ __forceinline__ void put(typename Elem<DT>::type *to, int c, const float (&v)[V]) const {
        if (whole(c))
            *reinterpret_cast<uint4 *>(to) = pack<DT>(v);
        else
            store_part<DT>(to, pack<DT>(v), lo(c), hi(c));
    }
};

// Rows from `first` on, `step` apart.
__device__ __forceinline__ int row_turns(int64_t M, int64_t first, int64_t step) {
    return first < M ? static_cast<int>((M - first + step - 1) / step) : 0;
}

// C chunks of every row per thread.  dw: in registers over all of the CTA's rows,
// then over the row slots in shared memory; one partial sum per CTA and column is
// left for mbt_rmsnorm_dw_finish_kernel.
template <int DT, int C, bool RES, bool PART, bool W32>
__global__ void __launch_bounds__(kRingThreads, 1)
    mbt_rmsnorm_backward_kernel(const __grid_constant__ NormGradArgs a, const __grid_constant__ RingArgs r) {
    using T = typename Elem<DT>::type;
    constexpr int V = Elem<DT>::kVec;
    extern __shared__ __align__(128) unsigned char dyn_smem[];
    __shared__ __align__(8) RingShared sh;
    ring_init(sh, r);
    RingState q(r, smem_u32(dyn_smem), smem_u32(&sh.bars[0]), WaitCtl{kDefaultWaitBudgetNs, &sh.abort_flag, r.status});
    q.start(r, a.M);
    const RingThread<DT, C, PART> th(r, a.M, a.N, q.ring);
    RingWeights<DT, C, PART, W32> wt;
    wt.load(r, a.w, a.wdt, a.woff, th.t, th.off, a.N);
    float dw[C][V];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < V; ++e) dw[c][e] = 0.f;
    const float inv_n = 1.f / static_cast<float>(a.N);
    const int64_t rows = static_cast<int64_t>(gridDim.x) * r.rows;   // from one row of a slot to the next
    T *dx = static_cast<T *>(a.dx) + th.first * a.ld_dx - th.off + th.t * V;
    const int chunk = r.tpr * V;
    int turn = 0;
    float next_rstd = th.first < a.M ? __ldg(a.rstd + th.first) : 0.f;
    const float *rstd_at = a.rstd + th.first;
    const int turns = row_turns(a.M, th.first - th.k % r.unit_rows, rows);
    const int mine = row_turns(a.M, th.first, rows);
    for (int n = 0; n < turns; ++n, dx += rows * a.ld_dx) {
        const uint32_t z1 = r.zero & n, z2 = r.zero & ~n;
        const float rstd = next_rstd;
        rstd_at += rows;
        if (n + 1 < mine) next_rstd = __ldg(rstd_at);
        q.wait();
        const int have = n < mine && q.alive ? th.count : 0;
        const int64_t i = PART ? th.first + n * rows : 0;   // (only parts of chunks ask for the row)
        uint4 vy[C], vh[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            vy[c] = vh[c] = make_uint4(0, 0, 0, 0);
            if (c >= have) continue;
            vy[c] = th.chunk(q.stage, 0, c);
            vh[c] = th.chunk(q.stage, 1, c);
        }
        if (PART && have && (th.head || th.tail))
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (th.whole(c)) continue;
                th.last_chunk(r, 0, c, i, vy[c]);
                th.last_chunk(r, 1, c, i, vh[c]);
                float f[V];
                unpack<DT>(vy[c], f);
                th.mask(c, f);
                vy[c] = pack<DT>(f);
                unpack<DT>(vh[c], f);
                th.mask(c, f);
                vh[c] = pack<DT>(f);
            }
        float dot = 0.f;
        uint32_t none = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float dy[V], h[V], w[V];
            unpack<DT>(vy[c], dy);
            unpack<DT>(vh[c], h);
            wt.get(c, z1, w);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float x = dy[e] * h[e];
                dot += x * w[e];
                dw[c][e] += x * rstd;
            }
        }
        row_reduce<false>(dot, none, r.tpr, sh.red[0], turn);
        turn ^= 1;
        // times h gives xh mean(g xh); from the sum on, as powers of rstd alone leave
        // fp32's range at rows that are themselves within it
        const float proj = rstd * (rstd * (dot * inv_n));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (c >= have) continue;
            uint4 vr = make_uint4(0, 0, 0, 0);
            if constexpr (RES) {
                vr = th.chunk(q.stage, 2, c);
                if (PART && th.tail) th.last_chunk(r, 2, c, i, vr);
            }
            float dy[V], h[V], d[V], f[V], w[V];
            unpack<DT>(again(vy[c], z2), dy);
            unpack<DT>(again(vh[c], z2), h);
            wt.get(c, z2, w);
            if constexpr (RES) unpack<DT>(vr, f);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                d[e] = rstd * (dy[e] * w[e] - h[e] * proj);
                if constexpr (RES) d[e] += f[e];
            }
            th.put(dx + c * chunk, c, d);
        }
        q.release(r, a.M);
    }
    q.drain(r.stages);
    if (!a.dw) return;
    // every stage has been read: its memory takes the row slots' sums
    float *slots = reinterpret_cast<float *>(dyn_smem);
    asm volatile("bar.sync 15, %0;" ::"n"(kRingThreads) : "memory");
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const int j = (th.t + c * r.tpr) * V + e - th.off;
            if (j >= 0 && j < a.N) slots[th.k * a.N + j] = dw[c][e];
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
        a.partial[blockIdx.x * a.N + j] = sum;
    }
}

template <int DT, int C, bool RES, bool Q, bool PART, bool W32>
__global__ void __launch_bounds__(kRingThreads, 1)
    mbt_rmsnorm_ring_kernel(const __grid_constant__ NormArgs a, const __grid_constant__ RingArgs r) {
    using T = typename Elem<DT>::type;
    using O = typename std::conditional<Q, uint8_t, T>::type;
    constexpr int V = Elem<DT>::kVec;
    extern __shared__ __align__(128) unsigned char dyn_smem[];
    __shared__ __align__(8) RingShared sh;
    ring_init(sh, r);
    RingState q(r, smem_u32(dyn_smem), smem_u32(&sh.bars[0]), WaitCtl{kDefaultWaitBudgetNs, &sh.abort_flag, r.status});
    q.start(r, a.M);
    const RingThread<DT, C, PART> th(r, a.M, a.N, q.ring);
    RingWeights<DT, C, PART, W32> wt;
    wt.load(r, a.w, a.wdt, a.woff, th.t, th.off, a.N);
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
            if (PART && have && th.tail)
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    th.last_chunk(r, 0, c, i, vx[c]);
                    if constexpr (RES) th.last_chunk(r, 1, c, i, vr[c]);
                }
#pragma unroll
            for (int c = 0; c < C; ++c) {
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
        if (PART && have && (th.head || th.tail))
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (!th.whole(c)) th.mask(c, h[c]);
        float ss = 0.f;
        uint32_t amax = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int e = 0; e < V; ++e) ss += h[c][e] * h[c][e];
            if (Q && a.quant == 0) {
                float w[V];
                wt.get(c, z2, w);
#pragma unroll
                for (int e = 0; e < V; ++e) w[e] *= h[c][e];
                amax = magnitude_max(amax, w);
            }
        }
        row_reduce<Q>(ss, amax, r.tpr, sh.red[0], turn);
        turn ^= 1;
        const float rstd = rsqrtf(ss * inv_n + a.eps);
        float scale = 0.f;
        Divisor by;
        if (Q && a.quant == 0) {
            scale = group_scale(magnitude(__uint_as_float(amax) * rstd));
            by = Divisor(scale);
        }
        if (th.t == 0 && n < mine) {
            a.rstd[i] = rstd;
            if (Q && a.quant == 0) a.scales[i] = scale;
        }
        uint32_t gmax[C];                    // largest magnitude of each chunk's group
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (c < have && write_res) th.put(res + c * chunk, c, h[c]);
            float w[V];
            wt.get(c, z1, w);
            const Pair rr(rstd);
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const float2 y = (Pair(h[c][e], h[c][e + 1]) * rr * Pair(w[e], w[e + 1])).get();
                h[c][e] = y.x, h[c][e + 1] = y.y;
            }
            if constexpr (!Q) {
                if (c < have) th.put(out + c * chunk, c, h[c]);
            } else if (a.quant > 0) {        // (rows start at a chunk)
                gmax[c] = magnitude_max(0u, h[c]);
            }
        }
        if constexpr (Q) {
            if (a.quant > 0) {
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
    auto term = [&](int64_t i) {
        return Elem<DT>::widen(static_cast<const T *>(a.dy)[i * a.ld_dy + j]) *
               (Elem<DT>::widen(static_cast<const T *>(a.h)[i * a.ld_h + j]) * a.rstd[i]);
    };
    float sum = 0.f;
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        float part[4] = {};
        const int n = static_cast<int>(min(hi - i0, int64_t{32}));
        int i = 0;
        for (; i + 16 <= n; i += 16)
#pragma unroll
            for (int k = 0; k < 16; ++k) part[k % 4] += term(i0 + i + k);
        for (; i + 4 <= n; i += 4)
#pragma unroll
            for (int k = 0; k < 4; ++k) part[k] += term(i0 + i + k);
        for (; i < n; ++i) part[0] += term(i0 + i);
        sum += pair_sum(part);
    }
    a.partial[s * a.N + j] = sum;
}

// dw from its partial sums: 32 columns a CTA, 16 threads a column, each adding
// every 16th split, four sums side by side, then the threads' in pairs.
constexpr int kFinishRows = 16;
__global__ void __launch_bounds__(32 * kFinishRows) mbt_rmsnorm_dw_finish_kernel(const NormGradArgs a) {
    __shared__ float part[kFinishRows][32];
    const int l = threadIdx.x & 31, s0 = threadIdx.x >> 5;
    const int64_t j = blockIdx.x * 32ll + l;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float sum[4] = {};
    if (j < a.N) {
#pragma unroll 10
        for (int64_t s = s0; s < a.splits; s += kFinishRows) {
            const float v = sum[0] + a.partial[s * a.N + j];
            sum[0] = sum[1], sum[1] = sum[2], sum[2] = sum[3], sum[3] = v;
        }
    }
    part[s0][l] = pair_sum(sum);
    __syncthreads();
    if (s0 != 0 || j >= a.N) return;
    float all[kFinishRows];
#pragma unroll
    for (int s = 0; s < kFinishRows; ++s) all[s] = part[s][l];
    a.dw[j] = pair_sum(all);
}

// Where the rows of a matrix start in 16-byte chunks: -1 if not known from the
// first row on, else the pitch's part beyond whole chunks (0: every row at a chunk).
int phase_of(const void *p, int64_t ld, int64_t es) {
    if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return -1;
    return static_cast<int>(ld * es % 16);
}

int weight_mode(const void *w, int wdt, int dtype) {
    if (!w) return kNoWeight;
    if (reinterpret_cast<uintptr_t>(w) % 16 != 0) return kAnyWeight;
    return wdt == dtype ? kSameWeight : wdt == MBT_F32 ? kF32Weight : kAnyWeight;
}

// Rows, threads, stages of a ring over these matrices.  False where it does not
// apply: rows too long for a CTA's registers or two stages, matrices whose rows
// start at different places in a chunk.  prefer: chunks a thread where the rows allow
// them (0: what was measured for this norm).
struct RingPlan {
    RingArgs r;
    int chunks;              // of 16 bytes per thread
    bool part;               // rows begin or end inside a chunk
    int grid, smem;
};

bool ring_plan(const void *const *in, const int64_t *ld, int inputs, int64_t M, int64_t N, int es, int ph,
               int most, int min_tpr, int sms, RingPlan *plan, int prefer = 0, int least = 2) {
    const int V = 16 / es;
    RingArgs &r = plan->r;
    r = RingArgs{};
    r.inputs = inputs;
    for (int i = 0; i < inputs; ++i) {
        r.in[i] = static_cast<const char *>(in[i]);
        r.ld[i] = ld[i] * es;
        r.tail[i] = first_tail_row(M, N * es, ld[i] * es);
    }
    r.phased = M > 1 && ph > 0;
    const int64_t chunks = (N + (r.phased ? V - 1 : 0) + V - 1) / V;
    // As many chunks a thread as its registers hold: rows side by side cost fewer
    // barriers than rows one after the other (bf16 4096 x 4096 gradient: 34.6 us
    // with 4 chunks, 50.3 with 1) ...
    const int usual = prefer ? prefer : most == 5 ? 4 : 32 / V;
    int tpr = min_tpr;
    while (tpr < kRingThreads && static_cast<int64_t>(tpr) * usual < chunks) tpr *= 2;
    if (static_cast<int64_t>(tpr) * most < chunks) return false;
    // ... but fewer rows at a time, by more threads each, until every CTA has a turn
    // (gradient of 64 x 4096: 9.6 us without, 6.7 with; waiting for four turns each
    // took 17.3 us against 15.9 of 1024 x 4096)
    while (tpr < kRingThreads && tpr < chunks && M * tpr < static_cast<int64_t>(sms) * kRingThreads) tpr *= 2;
    r.tpr = tpr;
    r.rows = kRingThreads / tpr;
    r.unit_threads = std::max(tpr, 32);
    r.unit_rows = r.unit_threads / tpr;
    r.row_bytes = static_cast<int32_t>(N * es);
    r.slot = static_cast<int32_t>((N * es + (r.phased ? 16 - es : 0) + 15) / 16 * 16);
    r.stage_bytes = static_cast<uint32_t>(r.slot) * r.unit_rows * inputs;
    const int64_t stage = static_cast<int64_t>(r.slot) * r.rows * inputs;
    r.stages = static_cast<int32_t>(std::min<int64_t>(kRingStages, kRingBytes / stage));
    if (r.stages < least) return false;
    plan->chunks = static_cast<int>((chunks + tpr - 1) / tpr);
    plan->part = r.phased || N % V != 0;
    plan->smem = static_cast<int>(std::max<int64_t>(r.stages * stage, r.rows * N * 4));
    const int64_t groups = (M + r.rows - 1) / r.rows;
    // a slot's rows, grid x rows apart, all start at the same place in a chunk
    plan->grid = static_cast<int>(std::min<int64_t>(groups, r.phased ? sms / 8 * 8 : sms));
    return plan->grid > 0;
}

template <class K, class A>
cudaError_t launch_ring(K kernel, const RingPlan &p, cudaStream_t s, const A &a) {
    // (set on every call: a kernel's limit is a property of the device it is loaded on)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    return launch_pipeline(kernel, p.grid, kRingThreads, p.smem, s, a, p.r);
}

// The kernel of a plan.  Whole chunks: the exact chunk count's class; parts of
// chunks: fewer classes (a thread's chunks past its own cost little beside the
// parts); fp32 weights of 16-bit rows: the largest class.
template <int DT, int C, bool PART, bool W32>
cudaError_t launch_ring_forward(const RingPlan &p, const NormArgs &a, cudaStream_t s) {
    const bool q = a.quant != MBT_QUANT_NONE;
    if (a.res)
        return q ? launch_ring(mbt_rmsnorm_ring_kernel<DT, C, true, true, PART, W32>, p, s, a)
                 : launch_ring(mbt_rmsnorm_ring_kernel<DT, C, true, false, PART, W32>, p, s, a);
    return q ? launch_ring(mbt_rmsnorm_ring_kernel<DT, C, false, true, PART, W32>, p, s, a)
             : launch_ring(mbt_rmsnorm_ring_kernel<DT, C, false, false, PART, W32>, p, s, a);
}

template <int DT, int C, bool PART, bool W32>
cudaError_t launch_ring_backward(const RingPlan &p, const NormGradArgs &a, cudaStream_t s) {
    return a.dres ? launch_ring(mbt_rmsnorm_backward_kernel<DT, C, true, PART, W32>, p, s, a)
                  : launch_ring(mbt_rmsnorm_backward_kernel<DT, C, false, PART, W32>, p, s, a);
}

template <int DT>
cudaError_t ring_forward(const RingPlan &p, const NormArgs &a, cudaStream_t s) {
    const int c = p.chunks;
    const bool part = p.part || p.r.wmode != kSameWeight;
    if constexpr (DT == MBT_F32) {
        if (part)
            return c <= 4   ? launch_ring_forward<DT, 4, true, false>(p, a, s)
                   : c <= 5 ? launch_ring_forward<DT, 5, true, false>(p, a, s)
                            : launch_ring_forward<DT, 8, true, false>(p, a, s);
        return c <= 2   ? launch_ring_forward<DT, 2, false, false>(p, a, s)
               : c <= 4 ? launch_ring_forward<DT, 4, false, false>(p, a, s)
                        : launch_ring_forward<DT, 8, false, false>(p, a, s);
    } else {
        if (p.r.wmode == kF32Weight || p.r.wmode == kAnyWeight)
            return launch_ring_forward<DT, 5, true, true>(p, a, s);
        if (part)
            return c <= 2   ? launch_ring_forward<DT, 2, true, false>(p, a, s)
                   : c <= 4 ? launch_ring_forward<DT, 4, true, false>(p, a, s)
                            : launch_ring_forward<DT, 5, true, false>(p, a, s);
        return c <= 1   ? launch_ring_forward<DT, 1, false, false>(p, a, s)
               : c <= 2 ? launch_ring_forward<DT, 2, false, false>(p, a, s)
               : c <= 4 ? launch_ring_forward<DT, 4, false, false>(p, a, s)
                        : launch_ring_forward<DT, 5, false, false>(p, a, s);
    }
}

template <int DT>
cudaError_t ring_backward(const RingPlan &p, const NormGradArgs &a, cudaStream_t s) {
    const int c = p.chunks;
    const bool part = p.part || p.r.wmode != kSameWeight;
    if constexpr (DT == MBT_F32) {
        if (part)
            return c <= 4 ? launch_ring_backward<DT, 4, true, false>(p, a, s)
                          : launch_ring_backward<DT, 5, true, false>(p, a, s);
        return c <= 2   ? launch_ring_backward<DT, 2, false, false>(p, a, s)
               : c <= 4 ? launch_ring_backward<DT, 4, false, false>(p, a, s)
                        : launch_ring_backward<DT, 5, false, false>(p, a, s);
    } else {
        if (p.r.wmode == kF32Weight || p.r.wmode == kAnyWeight)
            return launch_ring_backward<DT, 5, true, true>(p, a, s);
        if (part)
            return c <= 2   ? launch_ring_backward<DT, 2, true, false>(p, a, s)
                   : c <= 4 ? launch_ring_backward<DT, 4, true, false>(p, a, s)
                            : launch_ring_backward<DT, 5, true, false>(p, a, s);
        return c <= 1   ? launch_ring_backward<DT, 1, false, false>(p, a, s)
               : c <= 2 ? launch_ring_backward<DT, 2, false, false>(p, a, s)
               : c <= 4 ? launch_ring_backward<DT, 4, false, false>(p, a, s)
                        : launch_ring_backward<DT, 5, false, false>(p, a, s);
    }
}

cudaError_t launch_finish(const NormGradArgs &a, cudaStream_t s) {
    return launch_grid(mbt_rmsnorm_dw_finish_kernel, dim3(static_cast<unsigned>((a.N + 31) / 32)), 32 * kFinishRows, s, a);
}

// The gradient through the ring; *done says whether it applied.
template <int DT>
int backward_by_ring(NormGradArgs a, cudaStream_t s, int sms, bool *done) {
    constexpr int V = Elem<DT>::kVec, es = 16 / V;
    const int ph = phase_of(a.h, a.ld_h, es);
    bool same = ph >= 0 && phase_of(a.dy, a.ld_dy, es) == ph && phase_of(a.dx, a.ld_dx, es) == ph;
    if (a.dres) same = same && phase_of(a.dres, a.ld_dres, es) == ph;
    const void *in[3] = {a.dy, a.h, a.dres};
    const int64_t ld[3] = {a.ld_dy, a.ld_h, a.ld_dres};
    RingPlan p;
    *done = same && ring_plan(in, ld, a.dres ? 3 : 2, a.M, a.N, es, ph, 5, 8, sms, &p);
    if (!*done) return MBT_OK;
    int rc = device_status_word(&p.r.status);
    if (rc != MBT_OK) return rc;
    p.r.wmode = weight_mode(a.w, a.wdt, DT);
    a.splits = p.grid;
    WorkspaceHold hold;
    if (a.dw) {
        void *scratch = nullptr;
        rc = hold.scratch(s, static_cast<size_t>(a.splits) * a.N * 4, &scratch);
        if (rc != MBT_OK) return rc;
        a.partial = static_cast<float *>(scratch);
    }
    cudaError_t e = ring_backward<DT>(p, a, s);
    if (e == cudaSuccess && a.dw) e = launch_finish(a, s);
    return e == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
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

// Where the ring is faster than a row in registers (us, ring / registers, bf16 with a
// residual, both built and timed in turn):
//  - its start (weights, barriers, the first rows' latency) is paid once per call:
//    512 x 8192 7.95 / 7.87, 1024 x 8192 12.4 / 13.6, fp16 16384 x 16384 358 / 426;
//  - rows of up to 1 KB are a warp's at most in registers, with no barrier:
//    131072 x 256 46.5 / 41.0, 131072 x 512 91 / 80; fp32 65536 x 512 45 / 61;
//  - two matrices read keep enough bytes on their way with short rows as well:
//    65536 x 2048 183 / 160, 4096 x 4096 22.5 / 25.8; rows that start inside a
//    chunk do not: 65537 x 1001 105 / 127; nor does the arithmetic of an 8-bit
//    output, by groups of 128 65536 x 2048 202 / 238, 131072 x 1024 191 / 241.
bool ring_forward_pays(const NormArgs &a, int64_t es, int sms, int phase) {
    const int64_t row = a.N * es;
    if (a.M * row < (16ll << 20) || a.M < 4 * sms || row <= 1024) return false;
    return row > 4096 || !a.res || phase != 0 || a.quant != MBT_QUANT_NONE;
}

template <int DT>
cudaError_t forward_any(const NormArgs &a, cudaStream_t s) {
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
    RingPlan p;
    if (same && ring_forward_pays(a, es, sms, ph) &&
        ring_plan(in, ld, a.res ? 2 : 1, a.M, a.N, es, ph, V == 8 ? 5 : 8, a.quant > 0 ? 32 : 8, sms, &p)) {
        if (device_status_word(&p.r.status) != MBT_OK) return cudaErrorUnknown;
        p.r.wmode = weight_mode(a.w, a.wdt, DT);
        return ring_forward<DT>(p, a, s);
    }
    NormVecArgs va{a, 0, 0, a.M > 1 && ph > 0};
    const int64_t chunks = (a.N + (va.phased ? V - 1 : 0) + V - 1) / V;
    if (!same || chunks > 4 * 1024) {
        const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.M, 1 << 20)));
        return launch_grid(mbt_rmsnorm_rows_kernel<DT>, grid, kRowThreads, s, a);
    }
    // One chunk a thread where all rows then fit the device at once (at 1024
    // threads an SM), as the time is one row's latency: bf16 600 x 2048 2.6 us against
    // 2.9 with two.  Else two, as long as that keeps a row within a CTA: 256 x 8192 3.6
    // us against 5.3 with one and 4.2 with four.  A warp at least where groups of up
    // to 128 columns are reduced.
    int tpr = a.quant > 0 ? 32 : 8;
    while (tpr < 1024 && (tpr * 2 < chunks || (tpr < chunks && a.M * tpr * 2 <= 1024ll * sms))) tpr *= 2;
    va.tpr = tpr;
    va.wmode = weight_mode(a.w, a.wdt, DT);
    const int threads = tpr > 32 ? tpr : 128, rows = threads / tpr;
    if ((a.M + rows - 1) / rows > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>((a.M + rows - 1) / rows));
    const int64_t c = (chunks + tpr - 1) / tpr;
    return c <= 1   ? launch_forward<DT, 1>(va, grid, threads, s)
           : c <= 2 ? launch_forward<DT, 2>(va, grid, threads, s)
                    : launch_forward<DT, 4>(va, grid, threads, s);
}

// Any strides and lengths: column sums of dw in splits of rows, then dx, which may
// overwrite dy (bf16 2048 x 32768, residual, too long for the ring: 422 us, 1.3 TB/s).
template <int DT>
int backward_any(NormGradArgs a, cudaStream_t s) {
    int sms = 0, smem = 0;
    int rc = device_limits(&sms, &smem);
    if (rc != MBT_OK) return rc;
    bool done = false;
    rc = backward_by_ring<DT>(a, s, sms, &done);
    if (rc != MBT_OK || done) return rc;
    const int64_t cols = (a.N + kColThreads - 1) / kColThreads;
    if (a.dw) {
        // enough CTAs of 128 columns to fill the device, at least 32 rows each
        a.splits = std::max<int64_t>(1, std::min<int64_t>((a.M + 31) / 32, 16 * sms / cols));
        a.splits = std::min<int64_t>(a.splits, 65535);
        WorkspaceHold hold;
        void *scratch = nullptr;
        rc = hold.scratch(s, static_cast<size_t>(a.splits) * a.N * 4, &scratch);
        if (rc != MBT_OK) return rc;
        a.partial = static_cast<float *>(scratch);
        const dim3 grid(static_cast<unsigned>(cols), static_cast<unsigned>(a.splits));
        cudaError_t e = launch_grid(mbt_rmsnorm_dw_rows_kernel<DT>, grid, kColThreads, s, a);
        if (e == cudaSuccess) e = launch_finish(a, s);
        if (e != cudaSuccess) return MBT_ERR_CUDA;
    }
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(a.M, 1 << 20)));
    return launch_grid(mbt_rmsnorm_dx_rows_kernel<DT>, grid, kRowThreads, s, a) == cudaSuccess ? MBT_OK
                                                                                              : MBT_ERR_CUDA;
}

}  // namespace

template <int DT>
cudaError_t norm_forward(const NormArgs &a, cudaStream_t s) { return forward_any<DT>(a, s); }
template <int DT>
int norm_backward(const NormGradArgs &a, cudaStream_t s) { return backward_any<DT>(a, s); }

}  // namespace mbt
