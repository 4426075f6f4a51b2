// Element types of the layer operators: 16-byte vectors of fp16, bf16 or fp32
// widened exactly to fp32 and rounded back to nearest even, e4m3 pairs, and the
// reductions a row needs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "mbtile.h"

namespace mbt {
namespace {

constexpr float kE4m3Max = 448.f;
// Smallest scale of an 8-bit group: a group of zeros divides by it, not by 0.
constexpr float kMinScale = 1.17549435e-38f;   // 2^-126

template <int DT>
struct Elem;
template <>
struct Elem<MBT_F16> {
    using type = __half;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float widen(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half round(float v) { return __float2half_rn(v); }
    static __device__ __forceinline__ float2 widen2(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
    static __device__ __forceinline__ uint32_t round2(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
template <>
struct Elem<MBT_BF16> {
    using type = __nv_bfloat16;
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
    static __device__ __forceinline__ float2 widen2(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t round2(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};
template <>
struct Elem<MBT_F32> {
    using type = float;
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float widen(float v) { return v; }
    static __device__ __forceinline__ float round(float v) { return v; }
};

// A 16-byte vector as fp32 values, and back.
template <int DT>
__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[Elem<DT>::kVec]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == MBT_F32) {
            f[i] = __uint_as_float(w[i]);
        } else {
            const float2 p = Elem<DT>::widen2(w[i]);
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        }
    }
}

template <int DT>
__device__ __forceinline__ uint4 pack(const float (&f)[Elem<DT>::kVec]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (DT == MBT_F32)
            w[i] = __float_as_uint(f[i]);
        else
            w[i] = Elem<DT>::round2(f[2 * i], f[2 * i + 1]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Element i of an array whose type is known at run time only.
__device__ __forceinline__ float load_any(const void *p, int dtype, int64_t i) {
    if (dtype == MBT_F16) return __half2float(static_cast<const __half *>(p)[i]);
    if (dtype == MBT_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    return static_cast<const float *>(p)[i];
}

__device__ __forceinline__ void store_any(void *p, int dtype, int64_t i, float v) {
    if (dtype == MBT_F16)
        static_cast<__half *>(p)[i] = __float2half_rn(v);
    else if (dtype == MBT_BF16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float *>(p)[i] = v;
}

// Two values rounded to e4m3 (nearest even, saturating; NaN stays NaN): a in
// the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Two e4m3 values (low byte first) as an fp16 pair, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t v) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(v)));
    return r;
}

// Two fp32 values in one instruction, each rounded as alone.
struct Pair {
    uint64_t v;
    __device__ __forceinline__ Pair() {}
    __device__ __forceinline__ Pair(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    explicit __device__ __forceinline__ Pair(float a) : Pair(a, a) {}
    __device__ __forceinline__ float2 get() const {
        float2 f;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
        return f;
    }
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

// a / b rounded to nearest: b's reciprocal rounded to nearest and one correction
// (Markstein, IBM J. Res. Dev. 34, 1990).  nb = -b, ib = 1 / b.
__device__ __forceinline__ Pair divide(Pair a, Pair nb, Pair ib) {
    const Pair q = a * ib;
    return fma2(fma2(q, nb, a), ib, q);
}

// |v| as an integer that orders as the magnitude does, with NaN above infinity:
// the largest magnitude of a group is then NaN if any value is.
__device__ __forceinline__ uint32_t magnitude(float v) {
    return __float_as_uint(v) & 0x7fffffffu;
}

// The largest magnitude of m (one already) and the values of f, two at a time.
template <int V>
__device__ __forceinline__ uint32_t magnitude_max(uint32_t m, const float (&f)[V]) {
    float r = __uint_as_float(m);
#pragma unroll
    for (int e = 0; e < V; e += 2) asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(r), "f"(f[e]), "f"(f[e + 1]));
    return __float_as_uint(r);
}

// The scale of a group from its largest magnitude (NaN stays NaN).
__device__ __forceinline__ float group_scale(uint32_t amax) {
    const float s = __uint_as_float(amax) * (1.f / kE4m3Max);
    return s < kMinScale ? kMinScale : s;
}

// Division by a group's scale: minus the quotient rounded to nearest, as divide()
// has it, but that a zero keeps its sign.  (An infinite scale is left out of the
// correction, which would be infinity times 0 for the group's finite values.)
struct Divisor {
    float scale = 0.f, minus_inv = 0.f;
    Divisor() = default;
    explicit __device__ __forceinline__ Divisor(float s) {
        scale = s < __uint_as_float(0x7f800000u) ? s : 0.f;
        minus_inv = -__frcp_rn(s);
    }
    __device__ __forceinline__ float2 minus(float a, float b) const {
        const Pair y(a, b), mi(minus_inv), mq = y * mi;
        return fma2(fma2(mq, Pair(scale), y), mi, mq).get();
    }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace
}  // namespace mbt
