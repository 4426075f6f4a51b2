// tile_w4_matvec for one to four rows of x and a q of few elements: one kernel
// that reads q once and multiplies in fp32.  The tensor form (mbtile_w4.cu) needs x
// converted by a kernel before it and, with K sliced, its sums added by one after
// it, which it takes 3 to 4 us to make up for; with more elements or more rows of x
// its instructions win (few_pays has both sides).  1 row, 4096 x 4096: 5.9 us with q
// from device memory, 5.2 from L2, of which half is the start of the kernel and the latency of its reads, half
// instructions (4.6 an element, half of which are not arithmetic: addresses, x
// through shared memory, sums over lanes).
#pragma once

namespace mbt {
namespace {

constexpr int kFewTokens = 4;       // rows of x, at most
constexpr int kFewRows = 4;         // rows of q per warp
constexpr int kFewWarps = 4;
constexpr int kFewChunk = 1024;     // columns a warp takes at a time, 32 per lane

__device__ __forceinline__ uint4 load_q(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Nibble I (0..3) of w in the mantissa of 2^23 (`top`, in a register): 2^23 + 16^I value.
template <int I>
__device__ __forceinline__ float few_nibble(uint32_t w, uint32_t top) {
    float f;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=f"(f) : "r"(w), "n"(0xf << (4 * I)), "r"(top));
    return f;
}

// A warp takes 1024 columns of four rows of q at a time, a lane 32 adjacent ones of
// each (one 16-byte access, within one group of any size); the warps of a CTA share
// the rows' columns, or, of short rows, take rows of their own.  The warp's part
// of x passes through shared memory, where the pieces a lane reads lie in other
// banks than its neighbours'.  A value of q is had as fp32 from the mantissa of
// 2^23 by one multiplication and addition (v 16^-i - (2^23 16^-i + z), exact), two
// of them in one instruction, and multiplied with x in fp32; a lane's sum over its
// 32 columns is then multiplied by their scales.
template <int T, int XDT>
__global__ void __launch_bounds__(32 * kFewWarps, T == 1 ? 6 : T == 2 && XDT != MBT_E4M3 ? 5 : T <= 3 ? 4 : 3)
    mbt_w4_few_kernel(const __grid_constant__ W4Args a) {
    constexpr int kPieces = XDT == MBT_E4M3 ? 2 : 4;    // 16-byte pieces of a lane's part of a row of x
    constexpr int kCols = 32 / kPieces;
    __shared__ uint4 xs[kFewWarps][T][32 * kPieces];
    __shared__ float red[kFewWarps][kFewRows * T];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = a.few_split, part = warp % split, set = warp / split, sets = kFewWarps / split;
    const int64_t n0 = min((static_cast<int64_t>(blockIdx.x) * sets + set) * kFewRows, a.N - 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float acc[kFewRows][T];
#pragma unroll
    for (int r = 0; r < kFewRows; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t) acc[r][t] = 0.f;
    uint32_t top;   // (not known to the compiler, which would move it in every time)
    asm volatile("mov.b32 %0, 0x4b000000;" : "=r"(top));
    const Pair mul01(1.f, 0.0625f), mul23(0.00390625f, 0.000244140625f);
    // rows past the last one are the last one again
    const int rows = static_cast<int>(min(a.N - n0, static_cast<int64_t>(kFewRows)));
    const uint32_t K = static_cast<uint32_t>(a.K), groups = static_cast<uint32_t>(a.groups);
    for (uint32_t base = part * kFewChunk; base < K; base += split * kFewChunk) {
        const uint32_t col = base + 32 * lane;
        const bool in = col < K;
        uint4 q[kFewRows];
        float s[kFewRows];
        uint32_t zero[kFewRows];
        int64_t at[kFewRows];
        const uint8_t *pq = a.q + n0 * a.ld_q + col / 2;
        int64_t cell = n0 * groups + (col >> a.group_shift);
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) {
            q[r] = in ? load_q(pq) : make_uint4(0, 0, 0, 0);
            at[r] = cell;
            zero[r] = 8;
            if (r + 1 < rows) pq += a.ld_q, cell += groups;
        }
        if (a.sdt == MBT_F32) {
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) s[r] = in ? static_cast<const float *>(a.s)[at[r]] : 0.f;
        } else {
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
                const uint16_t b = in ? static_cast<const uint16_t *>(a.s)[at[r]] : 0;
                s[r] = a.sdt == MBT_BF16 ? __uint_as_float(static_cast<uint32_t>(b) << 16)
                                         : __half2float(__ushort_as_half(b));
            }
        }
        if (a.z) {
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) zero[r] = in ? a.z[at[r]] : 8;
        }
        // (warp-uniform) x, piece by piece
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int piece = 32 * i + lane;
                const uint32_t col = base + piece * kCols;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (col < K)
                    v = *reinterpret_cast<const uint4 *>(static_cast<const unsigned char *>(a.x) +
                                                         (t * a.ld_x + col) * (16 / kCols));
                xs[warp][t][piece ^ ((piece >> 3) & (kPieces - 1))] = v;
            }
        float down[T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
            down[t] = 1.f;
            if (XDT == MBT_E4M3 && !a.x_row_scale && in)
                down[t] = a.xs[t * a.x_groups + col / 128];
        }
        __syncwarp();
        Pair add01[kFewRows], add23[kFewRows], p[kFewRows][T];
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) {
            const float bias = __uint_as_float((zero[r] & 15u) | 0xcb000000u), z = bias + 8388608.f;   // -(2^23 + z), -z
            add01[r] = Pair(bias, z - 524288.f);
            add23[r] = Pair(z - 32768.f, z - 2048.f);
#pragma unroll
            for (int t = 0; t < T; ++t) p[r][t] = Pair(0.f);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            Pair x[T][4];
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const int piece = lane * kPieces + j * kPieces / 4;
                const uint4 *at = &xs[warp][t][piece ^ ((piece >> 3) & (kPieces - 1))];
                uint32_t v[4];
                if constexpr (XDT == MBT_E4M3) {
                    const uint2 w = reinterpret_cast<const uint2 *>(at)[j & 1];
                    v[0] = e4m3x2_to_half2(w.x), v[1] = e4m3x2_to_half2(w.x >> 16);
                    v[2] = e4m3x2_to_half2(w.y), v[3] = e4m3x2_to_half2(w.y >> 16);
                } else {
                    const uint4 w = *at;
                    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 f = Elem<XDT == MBT_BF16 ? MBT_BF16 : MBT_F16>::widen2(v[k]);
                    x[t][k] = Pair(f.x, f.y);
                }
            }
#pragma unroll
            for (int r = 0; r < kFewRows; ++r) {
                const uint32_t w = j == 0 ? q[r].x : j == 1 ? q[r].y : j == 2 ? q[r].z : q[r].w, h = w >> 16;
                const Pair d[4] = {fma2(Pair(few_nibble<0>(w, top), few_nibble<1>(w, top)), mul01, add01[r]),
                                   fma2(Pair(few_nibble<2>(w, top), few_nibble<3>(w, top)), mul23, add23[r]),
                                   fma2(Pair(few_nibble<0>(h, top), few_nibble<1>(h, top)), mul01, add01[r]),
                                   fma2(Pair(few_nibble<2>(h, top), few_nibble<3>(h, top)), mul23, add23[r])};
#pragma unroll
                for (int t = 0; t < T; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) p[r][t] = fma2(d[k], x[t][k], p[r][t]);
            }
        }
#pragma unroll
        for (int r = 0; r < kFewRows; ++r)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const float2 v = p[r][t].get();
                acc[r][t] += (v.x + v.y) * down[t] * s[r];
            }
        __syncwarp();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
    for (int r = 0; r < kFewRows; ++r)
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const float v = warp_sum(acc[r][t]);
            if (lane == 0) red[warp][r * T + t] = v;
        }
    __syncthreads();
    // the parts' sums in order
    const int i = threadIdx.x;
    if (i >= sets * kFewRows * T) return;
    const int of = i / (kFewRows * T), r = i % (kFewRows * T) / T, t = i % T;
    const int64_t n = (static_cast<int64_t>(blockIdx.x) * sets + of) * kFewRows + r;
    if (n >= a.N) return;
    float y = 0.f;
    for (int k = 0; k < split; ++k) y += red[of * split + k][r * T + t];
    if (XDT == MBT_E4M3 && a.x_row_scale) y *= a.xs[t];
    store_any(a.out, a.odt, t * a.ld_out + n, y);
}

// Where the fp32 form takes less time than the tensor form; us, bf16 x, groups of 128,
// q from device memory, fp32 / tensor:
//                 4096 x 4096   8192 x 8192   16384 x 16384
//   1 row of x    5.9 /  8.7    14.4 / 14.8    45.1 / 37.4
//   2 rows        7.4 /  8.8    19.3 / 15.0    63.9 / 37.4
//   3 rows        8.5 /  9.0    23.2 / 15.1    77.3 / 37.6
//   4 rows       11.2 /  9.0    29.6 / 15.1   100.9 / 37.7
// and at 1024 x 1024 from 2.0 / 5.2 (1 row) to 2.6 / 5.5 (4 rows).
bool few_pays(int64_t T, int64_t N, int64_t K) {
    return T <= kFewTokens && N * K <= (T == 1 ? 96ll << 20 : (48ll << 20) / T);
}

template <int XDT>
cudaError_t launch_few(const W4Args &a, dim3 grid, cudaStream_t s) {
    constexpr int threads = 32 * kFewWarps;
    return a.T == 1   ? launch_grid(mbt_w4_few_kernel<1, XDT>, grid, threads, s, a)
           : a.T == 2 ? launch_grid(mbt_w4_few_kernel<2, XDT>, grid, threads, s, a)
           : a.T == 3 ? launch_grid(mbt_w4_few_kernel<3, XDT>, grid, threads, s, a)
                      : launch_grid(mbt_w4_few_kernel<4, XDT>, grid, threads, s, a);
}

}  // namespace
}  // namespace mbt
