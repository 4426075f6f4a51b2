// tile_adamw: one AdamW step over many tensors.
//
//   m' = b1 m + (1 - b1) g          v' = b2 v + (1 - b2) g^2
//   p' = p (1 - lr wd) - (lr / bc1) m' / (sqrt(v') / sqrt(bc2) + eps)
//
// with bc = 1 - b^step, all in fp32.  Every element is read and written once,
// so the bound with fp32 states is device memory (28 bytes an element in fp32:
// 100 M elements 398 us, 7.0 TB/s; bf16 with an fp32 master copy, 40 M: 168 us,
// 6.7 TB/s).  A launch takes a table of tensors as a kernel parameter (no upload,
// nothing kept between calls); a CTA finds its chunk's tensor in the table's
// running chunk counts.  A chunk is two 8-element accesses of each thread, all
// of whose loads are under way before the first is used: with one, each CTA's
// search and start are paid twice as often (8-bit states, 300 M bf16: 1.6
// times the time), and a loop over more chunks in a CTA leaves the memory idle
// between them (819).
//
// 8-bit states: blocks of 256 elements share an fp32 scale; one warp holds a
// block (8 elements a lane), so a block's largest magnitude is one warp
// reduction.  m is rounded to nearest e4m3.  sqrt(v) is stored instead of v
// (half the exponent range) and rounded up or down at random: with b2 near 1 a
// step changes v by less than half a code, and nearest rounding would leave it
// where it is for ever.  The random bits are a hash of (seed, tensor, element),
// so a call is reproducible.  sqrt(v) > 0 is never stored as 0, or m / sqrt(v)
// of the next step could be as large as m / eps.
#include "internal.h"
#include "mbtile_elem.cuh"
#include "mbtile_ptx.cuh"

namespace mbt {
namespace {

constexpr int kAdamThreads = 256;
constexpr int kAdamBlock = 256;                  // elements that share a scale
constexpr int kAdamChunk = kAdamThreads * 8 * 2; // elements a CTA updates
// A launch's parameters hold at most 32764 bytes; calls of few tensors take the
// small table, whose launch has less to send (8 tensors, 100,000 elements in all: 3.5 us
// against 4.6).
constexpr int kAdamSmallTable = 32;
constexpr int kAdamLargeTable = 440;

struct AdamTensor {
    void *p;
    const void *g;
    void *m, *v;
    float *w, *ms, *vs;
    int64_t n;
};

struct AdamScalars {
    float decay;       // 1 - lr wd
    float step_size;   // lr / bc1
    float inv_bc2;     // 1 / sqrt(bc2)
    float eps;
    float b1, b2, c1, c2;   // c = 1 - b
    float minus_zero;  // -0, not known to the compiler
    const float *grad_scale;
    uint32_t seed;
    int32_t pdt, gdt;  // element types of parameters and gradients
    int32_t first;     // index of the table's first tensor in the call
    int32_t count;
};

template <int TABLE>
struct AdamTable {
    AdamScalars s;
    AdamTensor t[TABLE];
    uint32_t end[TABLE];      // chunks up to and with tensor k
    uint32_t aligned[(TABLE + 31) / 32];   // tensors whose arrays allow vector access
};

// The 32-bit finaliser of MurmurHash3 (public domain).
__device__ __forceinline__ uint32_t mix32(uint32_t h) {
    h = (h ^ (h >> 16)) * 0x85EBCA6Bu;
    h = (h ^ (h >> 13)) * 0xC2B2AE35u;
    return h ^ (h >> 16);
}

// 16 random bits r as what is added to a value's mantissa: r 2^4 + 2^3.
__device__ __forceinline__ uint32_t dither_low(uint32_t h) { return (h << 4 & 0xFFFF0u) | 8u; }
__device__ __forceinline__ uint32_t dither_high(uint32_t h) { return (h >> 12 & 0xFFFF0u) | 8u; }

// t >= 0 rounded to a multiple of its e4m3 spacing, up with the probability of
// the part cut off: 20 mantissa bits are cut, 16 of them compared with the dither's.
// Below 2^-6 the spacing is that of 2^-6, which adding 2^-6 gives.
__device__ __forceinline__ float round_at_random(float t, uint32_t dither) {
    const float low = t < 0.015625f ? 0.015625f : 0.f;
    const uint32_t b = __float_as_uint(t + low) + dither;
    const float y = __uint_as_float(b & ~0xFFFFFu) - low;
    return t > 0.f ? fmaxf(y, 0.001953125f) : t;
}

__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Eight consecutive values (wide: fp32, else 16-bit of type dt) at p, 16-byte aligned.
template <bool WIDE>
struct Raw8 {
    uint4 a, b;
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        if constexpr (WIDE) {
            const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i);
            a = q[0];
            b = q[1];
        } else {
            a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8], int dt) const {
        if constexpr (WIDE) {
            f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y);
            f[2] = __uint_as_float(a.z), f[3] = __uint_as_float(a.w);
            f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y);
            f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
        } else if (dt == MBT_BF16) {
            unpack<MBT_BF16>(a, f);
        } else {
            unpack<MBT_F16>(a, f);
        }
    }
};

template <bool WIDE>
__device__ __forceinline__ void put8(void *p, int64_t i, const float (&f)[8], int dt) {
    if constexpr (WIDE) {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        const uint4 v = dt == MBT_BF16 ? pack<MBT_BF16>(f) : pack<MBT_F16>(f);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + i) = v;
    }
}

__device__ __forceinline__ void e4m3x8_get(const uint2 &q, float scale, float (&f)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t w = (k < 2 ? q.x : q.y) >> (16 * (k & 1));
        const float2 h = Elem<MBT_F16>::widen2(e4m3x2_to_half2(w)), v = (Pair(h.x, h.y) * Pair(scale)).get();
        f[2 * k] = v.x;
        f[2 * k + 1] = v.y;
    }
}

__device__ __forceinline__ uint2 e4m3x8_put(const float (&f)[8]) {
    uint2 q;
    q.x = to_e4m3x2(f[0], f[1]) | to_e4m3x2(f[2], f[3]) << 16;
    q.y = to_e4m3x2(f[4], f[5]) | to_e4m3x2(f[6], f[7]) << 16;
    return q;
}

// New p, m and v of eight elements, states in fp32.  sqrt and division to 1 and 2
// ulp: only p sees them.
__device__ __forceinline__ void update32(const AdamScalars &s, float gscale, float (&p)[8],
                                         const float (&g)[8], float (&m)[8], float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float gk = g[k] * gscale;
        m[k] = s.b1 * m[k] + s.c1 * gk;
        v[k] = s.b2 * v[k] + s.c2 * gk * gk;
        p[k] = s.decay * p[k] - s.step_size * __fdividef(m[k], sqrt_approx(v[k]) * s.inv_bc2 + s.eps);
    }
}

__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// New p and 8-bit states of a block, eight elements a lane: m and v come in as
// values, m and root leave as codes' values, ms and vs as scales.  Every operation
// of the states is rounded by itself, as the formulas read, so that the codes do
// not depend on how products and sums are fused.  Packed pairs halve the
// arithmetic, which is what bounds this form: about 68 instructions an element
// with the loads, hash and conversions, against 10 bytes of bf16 parameters,
// gradients and states (300 M elements: 657 us, 4.6 TB/s, with 79 % of the issue
// slots taken, some of them by values kept in local memory, see below; with fp32
// parameters and gradients, 16 bytes, 100 M: 254 us, 6.3 TB/s).
__device__ __forceinline__ void update8(const AdamScalars &s, float gscale, float (&p)[8], const float (&g)[8],
                                        float (&m)[8], float (&v)[8], float (&root)[8], const uint32_t (&r)[8],
                                        float *ms, float *vs) {
    Pair mp[4], vp[4];
    const Pair b1(s.b1), c1(s.c1), b2(s.b2), c2(s.c2), gs(gscale);
    // Products that are summed must not be fused with the sum, which the assembler
    // does with packed ones: fused with an addend of -0 that it does not know.
    const Pair zero(s.minus_zero);
    uint32_t am = 0, av = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const Pair gp = Pair(g[2 * k], g[2 * k + 1]) * gs;
        mp[k] = fma2(b1, Pair(m[2 * k], m[2 * k + 1]), zero) + fma2(c1, gp, zero);
        vp[k] = fma2(b2, Pair(v[2 * k], v[2 * k + 1]), zero) + fma2(c2 * gp, gp, zero);
        const float2 a = mp[k].get(), b = vp[k].get();
        const float af[2] = {a.x, a.y}, bf[2] = {b.x, b.y};
        am = magnitude_max(am, af);
        av = magnitude_max(av, bf);
    }
    am = __reduce_max_sync(0xffffffffu, am);
    av = __reduce_max_sync(0xffffffffu, av);
    *ms = group_scale(am);
    *vs = group_scale(magnitude(__fsqrt_rn(__uint_as_float(av))));   // (the largest root is the largest's)
    if (max(am, av) >= 0x7f800000u) {
        // an infinity or NaN in the block: the plain functions
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
            float mk = 0.f, vk = 0.f, pk = 0.f;
            uint32_t rk = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 a = mp[i / 2].get(), b = vp[i / 2].get();
                if (i == k) mk = i & 1 ? a.y : a.x, vk = i & 1 ? b.y : b.x, pk = p[i], rk = r[i];
            }
            const float x = __fsqrt_rn(vk);
            pk = s.decay * pk - s.step_size * (mk / (x * s.inv_bc2 + s.eps));
            const float cm = __fdiv_rn(mk, *ms), cv = round_at_random(__fdiv_rn(x, *vs), rk);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i == k) p[i] = pk, m[i] = cm, root[i] = cv;
        }
        return;
    }
    const Pair nms(-*ms), ims(__frcp_rn(*ms)), nvs(-*vs), ivs(__frcp_rn(*vs));
    float least = kE4m3Max;
    const Pair half(0.5f), minus(-1.f), ibc(s.inv_bc2), eps(s.eps), decay(s.decay), step(-s.step_size);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        // sqrt from its reciprocal's approximation and one correction (Markstein, as
        // above); the smallest value above 0 stands for 0 in the reciprocal, which stays finite
        const float2 b = vp[k].get();
        const Pair y(rsqrt_approx(fmaxf(b.x, 1.4e-45f)), rsqrt_approx(fmaxf(b.y, 1.4e-45f)));
        const Pair x0 = vp[k] * y;
        const Pair x = fma2(fma2(x0 * minus, x0, vp[k]), y * half, x0);
        const float2 d = fma2(x, ibc, eps).get();
        const Pair up = mp[k] * Pair(rcp_approx(d.x), rcp_approx(d.y));
        const float2 np = fma2(up, step, Pair(p[2 * k], p[2 * k + 1]) * decay).get();
        p[2 * k] = np.x;
        p[2 * k + 1] = np.y;
        const float2 cm = divide(mp[k], nms, ims).get(), cv = divide(x, nvs, ivs).get();
        m[2 * k] = cm.x;
        m[2 * k + 1] = cm.y;
        root[2 * k] = cv.x;
        root[2 * k + 1] = cv.y;
        asm("min.f32 %0, %1, %2, %3;" : "=f"(least) : "f"(least), "f"(cv.x), "f"(cv.y));
    }
    // below the normal codes (2^-6: 1 / 28672 of the block's largest) the rounding
    // takes twice the instructions; blocks without such an element go without (300 M
    // bf16 elements: 5 % less time)
    if (__any_sync(0xffffffffu, least < 0.015625f)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) root[k] = round_at_random(root[k], r[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            root[k] = __uint_as_float((__float_as_uint(root[k]) + r[k]) & ~0xFFFFFu);
    }
}

// Four CTAs an SM: held to 64 registers the 8-bit forms keep a third more warps
// to cover each other's chains (fp32 100 M 15 % faster, bf16 300 M 1 %) for 92 to 136
// bytes a thread kept in local memory; five CTAs keep more there (8 % slower).
template <bool PWIDE, bool GWIDE, bool MASTER, bool STATE8, int TABLE>
__global__ void __launch_bounds__(kAdamThreads, 4)
    mbt_adamw_kernel(const __grid_constant__ AdamTable<TABLE> a) {
    const AdamScalars &s = a.s;
    // the chunk's tensor: the first whose running count is above the chunk
    int lo = 0, hi = s.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.end[mid] > blockIdx.x)
            hi = mid;
        else
            lo = mid + 1;
    }
    const AdamTensor &t = a.t[lo];
    const int64_t chunk = blockIdx.x - (lo ? a.end[lo - 1] : 0u);
    const bool vec = a.aligned[lo >> 5] >> (lo & 31) & 1u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t counter = static_cast<uint32_t>(s.first + lo) * 0x9E3779B9u;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float gscale = s.grad_scale ? *s.grad_scale : 1.f;
    const int64_t base0 = chunk * kAdamChunk + warp * kAdamBlock;
    constexpr int kRounds = kAdamChunk / (kAdamThreads * 8);
    const int64_t step = kAdamThreads * 8;
    if (vec && chunk * kAdamChunk + kAdamChunk <= t.n) {
        // whole chunk: every load of the CTA's rounds is under way before the first use
        Raw8<MASTER || PWIDE> p[kRounds];
        Raw8<GWIDE> g[kRounds];
        Raw8<true> m[kRounds], v[kRounds];
        uint2 m8[kRounds], v8[kRounds];
        float ms[kRounds], vs[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int64_t i = base0 + r * step + lane * 8;
            p[r].load(MASTER ? static_cast<const void *>(t.w) : t.p, i);
            g[r].load(t.g, i);
            if constexpr (STATE8) {
                m8[r] = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(t.m) + i);
                v8[r] = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(t.v) + i);
                ms[r] = t.ms[i / kAdamBlock];
                vs[r] = t.vs[i / kAdamBlock];
            } else {
                m[r].load(t.m, i);
                v[r].load(t.v, i);
            }
        }
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int64_t i = base0 + r * step + lane * 8;
            float fp[8], fg[8], fm[8], fv[8], root[8];
            p[r].get(fp, s.pdt);
            g[r].get(fg, s.gdt);
            if constexpr (STATE8) {
                e4m3x8_get(m8[r], ms[r], fm);
                e4m3x8_get(v8[r], vs[r], fv);
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                    const Pair x(fv[k], fv[k + 1]);
                    const float2 v = (x * x).get();
                    fv[k] = v.x, fv[k + 1] = v.y;
                }
            } else {
                m[r].get(fm, MBT_F32);
                v[r].get(fv, MBT_F32);
            }
            if constexpr (STATE8) {
                uint32_t rnd[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t h = mix32((counter + static_cast<uint32_t>(i / 2 + k)) ^ s.seed);
                    rnd[2 * k] = dither_low(h);
                    rnd[2 * k + 1] = dither_high(h);
                }
                float nms, nvs;
                update8(s, gscale, fp, fg, fm, fv, root, rnd, &nms, &nvs);
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(t.m) + i) = e4m3x8_put(fm);
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(t.v) + i) = e4m3x8_put(root);
                if (lane == 0) {
                    t.ms[i / kAdamBlock] = nms;
                    t.vs[i / kAdamBlock] = nvs;
                }
            } else {
                update32(s, gscale, fp, fg, fm, fv);
                put8<true>(t.m, i, fm, MBT_F32);
                put8<true>(t.v, i, fv, MBT_F32);
            }
            if constexpr (MASTER) put8<true>(t.w, i, fp, MBT_F32);
            put8<PWIDE>(t.p, i, fp, s.pdt);
        }
        return;
    }
    // a tensor's end, or arrays of any alignment: element by element, a lane's
    // eight elements 32 apart so that a warp's accesses are contiguous
    for (int r = 0; r < kRounds; ++r) {
        const int64_t base = base0 + r * step;
        if (base >= t.n) return;
        float fp[8], fg[8], fm[8], fv[8], root[8];
        float ms = 0.f, vs = 0.f;
        if constexpr (STATE8) {
            ms = t.ms[base / kAdamBlock];
            vs = t.vs[base / kAdamBlock];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t i = base + 32 * k + lane;
            const bool in = i < t.n;
            fp[k] = fg[k] = fm[k] = fv[k] = 0.f;
            if (!in) continue;
            fp[k] = MASTER ? t.w[i] : load_any(t.p, PWIDE ? MBT_F32 : s.pdt, i);
            fg[k] = load_any(t.g, GWIDE ? MBT_F32 : s.gdt, i);
            if constexpr (STATE8) {
                const float2 h = Elem<MBT_F16>::widen2(
                    e4m3x2_to_half2(static_cast<const uint8_t *>(t.m)[i] |
                                    static_cast<const uint8_t *>(t.v)[i] << 8));
                fm[k] = h.x * ms;
                fv[k] = h.y * vs;
                fv[k] *= fv[k];
            } else {
                fm[k] = static_cast<const float *>(t.m)[i];
                fv[k] = static_cast<const float *>(t.v)[i];
            }
        }
        if constexpr (STATE8) {
            // elements past the end have m = v = 0 and leave the block's scales alone
            uint32_t rnd[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int64_t i = base + 32 * k + lane;
                const uint32_t h = mix32((counter + static_cast<uint32_t>(i / 2)) ^ s.seed);
                rnd[k] = i & 1 ? dither_high(h) : dither_low(h);
            }
            float nms, nvs;
            update8(s, gscale, fp, fg, fm, fv, root, rnd, &nms, &nvs);
            if (lane == 0) {
                t.ms[base / kAdamBlock] = nms;
                t.vs[base / kAdamBlock] = nvs;
            }
        } else {
            update32(s, gscale, fp, fg, fm, fv);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t i = base + 32 * k + lane;
            if (i >= t.n) continue;
            if constexpr (MASTER) t.w[i] = fp[k];
            store_any(t.p, PWIDE ? MBT_F32 : s.pdt, i, fp[k]);
            if constexpr (STATE8) {
                const uint32_t c = to_e4m3x2(fm[k], root[k]);
                static_cast<uint8_t *>(t.m)[i] = static_cast<uint8_t>(c);
                static_cast<uint8_t *>(t.v)[i] = static_cast<uint8_t>(c >> 8);
            } else {
                static_cast<float *>(t.m)[i] = fm[k];
                static_cast<float *>(t.v)[i] = fv[k];
            }
        }
    }
}

template <int TABLE>
cudaError_t launch_table(const AdamTable<TABLE> &a, bool master, bool state8, uint32_t chunks,
                         cudaStream_t stream) {
    const bool pw = a.s.pdt == MBT_F32, gw = a.s.gdt == MBT_F32;
    void (*k)(const AdamTable<TABLE>) = nullptr;
#define MBT_ADAMW_PICK(P, G, W)                                         \
    if (pw == P && gw == G && master == W)                              \
        k = state8 ? mbt_adamw_kernel<P, G, W, true, TABLE>             \
                   : mbt_adamw_kernel<P, G, W, false, TABLE>;
    MBT_ADAMW_PICK(true, true, false)
    MBT_ADAMW_PICK(true, false, false)
    MBT_ADAMW_PICK(false, true, false)
    MBT_ADAMW_PICK(false, false, false)
    MBT_ADAMW_PICK(false, true, true)
    MBT_ADAMW_PICK(false, false, true)
#undef MBT_ADAMW_PICK
    return launch_pipeline(k, static_cast<int>(chunks), kAdamThreads, 0, stream, a);
}

bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

uintptr_t natural(int dtype) { return dtype == MBT_F32 ? 4 : 2; }

template <int TABLE>
int run_tables(const mbt_adamw_tensor *tensors, int64_t count, const AdamScalars &s, bool master,
               bool state8, cudaStream_t stream) {
    AdamTable<TABLE> a;
    a.s = s;
    int64_t k = 0;
    while (k < count) {
        uint64_t chunks = 0;
        int n = 0;
        a.s.first = static_cast<int32_t>(k);
        for (uint32_t &w : a.aligned) w = 0;
        for (; k < count && n < TABLE; ++k) {
            const mbt_adamw_tensor &t = tensors[k];
            const uint64_t c = static_cast<uint64_t>((t.n + kAdamChunk - 1) / kAdamChunk);
            if (chunks + c > 0x7fffffffull) break;
            chunks += c;
            a.t[n] = {t.param, t.grad, t.exp_avg, t.exp_avg_sq, t.master, t.m_scales, t.v_scales, t.n};
            a.end[n] = static_cast<uint32_t>(chunks);
            const uintptr_t st = state8 ? 8 : 16;
            if (aligned_to(t.param, 16) && aligned_to(t.grad, 16) && aligned_to(t.exp_avg, st) &&
                aligned_to(t.exp_avg_sq, st) && aligned_to(t.master, 16))
                a.aligned[n >> 5] |= 1u << (n & 31);
            ++n;
        }
        a.s.count = n;
        if (chunks == 0) continue;
        if (launch_table<TABLE>(a, master, state8, static_cast<uint32_t>(chunks), stream) !=
            cudaSuccess)
            return MBT_ERR_CUDA;
    }
    return MBT_OK;
}

}  // namespace
}  // namespace mbt

extern "C" int tile_adamw(const mbt_adamw_tensor *tensors, int64_t count, int param_dtype,
                          int grad_dtype, int state_dtype, int64_t step, double lr, double beta1,
                          double beta2, double eps, double weight_decay, const float *grad_scale,
                          uint32_t seed, void *stream) {
    using namespace mbt;
    if (count < 0 || (count > 0 && tensors == nullptr)) return MBT_ERR_ARG;
    if (param_dtype < MBT_F16 || param_dtype > MBT_F32 || grad_dtype < MBT_F16 ||
        grad_dtype > MBT_F32 || (state_dtype != MBT_F32 && state_dtype != MBT_E4M3))
        return MBT_ERR_ARG;
    if (step < 1 || !(lr >= 0.0) || !(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) ||
        !(eps >= 0.0) || !(weight_decay >= 0.0))
        return MBT_ERR_ARG;
    if (!aligned_to(grad_scale, 4)) return MBT_ERR_ALIGN;
    const bool state8 = state_dtype == MBT_E4M3;
    bool master = false, any = false;
    for (int64_t k = 0; k < count; ++k) {
        const mbt_adamw_tensor &t = tensors[k];
        if (t.n < 0 || t.n > (int64_t{1} << 40)) return MBT_ERR_ARG;
        if (t.n == 0) continue;
        if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return MBT_ERR_ARG;
        if (state8 ? !t.m_scales || !t.v_scales : t.m_scales || t.v_scales) return MBT_ERR_ARG;
        if (t.master && param_dtype == MBT_F32) return MBT_ERR_ARG;
        if (any && master != (t.master != nullptr)) return MBT_ERR_ARG;   // all or none
        master = t.master != nullptr;
        any = true;
        const uintptr_t st = state8 ? 1 : 4;
        if (!aligned_to(t.param, natural(param_dtype)) || !aligned_to(t.grad, natural(grad_dtype)) ||
            !aligned_to(t.exp_avg, st) || !aligned_to(t.exp_avg_sq, st) || !aligned_to(t.master, 4) ||
            !aligned_to(t.m_scales, 4) || !aligned_to(t.v_scales, 4))
            return MBT_ERR_ALIGN;
    }
    if (!any) return MBT_OK;
    AdamScalars s{};
    const double bc1 = 1.0 - pow(beta1, static_cast<double>(step));
    const double bc2 = 1.0 - pow(beta2, static_cast<double>(step));
    s.decay = static_cast<float>(1.0 - lr * weight_decay);
    s.step_size = static_cast<float>(lr / bc1);
    s.inv_bc2 = static_cast<float>(1.0 / sqrt(bc2));
    s.eps = static_cast<float>(eps);
    s.b1 = static_cast<float>(beta1);
    s.b2 = static_cast<float>(beta2);
    s.c1 = static_cast<float>(1.0 - beta1);
    s.c2 = static_cast<float>(1.0 - beta2);
    s.minus_zero = -0.f;
    s.grad_scale = grad_scale;
    s.seed = seed;
    s.pdt = param_dtype;
    s.gdt = grad_dtype;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return count <= kAdamSmallTable
               ? run_tables<kAdamSmallTable>(tensors, count, s, master, state8, st)
               : run_tables<kAdamLargeTable>(tensors, count, s, master, state8, st);
}
