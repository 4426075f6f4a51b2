// tile_grad_norm and tile_grad_scale: the norm of all elements of many tensors, the
// factor that clips it, and the product with a factor in place.
//
//   norm = |gs| (sum g^2)^(1/2)      scale = gs min(1, max_norm / (norm + eps))
//
// The norm reads every byte once, the product reads and writes it: device memory bounds
// both.  A launch takes a table of tensors as a kernel parameter.  The tensors' 16-byte
// vectors are cut into chunks of kGradVecs a thread; the norm's are dealt to a grid of whole
// CTAs per SM in spans, so that a CTA finds its first tensor once and steps to the next, and
// few sums are left to add up.  What lies before a tensor's first aligned vector and behind
// its last (at most 7 elements each) goes with its first chunk.  Calls of few chunks are
// one cluster, which also multiplies by the factor that it has found.
//
// A thread sums the squares of up to 64 chunks in fp32.  Where a chunk's sum leaves 2^-100 .. 2^100, in which
// squares neither overflow nor lose their last bits, it takes the chunk again in 64
// bits, so that the norm is right wherever fp32 holds it.  CTAs and threads are added in
// 64 bits in a fixed order, by the CTA that finishes last.  (bf16 300 M elements in 160 tensors:
// norm 89 us, 6.7 TB/s, product 172 us, 7.0 TB/s; 40 M in 96 tensors: 17.9 and 25.7 us.)
#include <algorithm>
#include <initializer_list>
#include <memory>
#include <new>

#include "mbtile_elem.cuh"
#include "mbtile_layer.h"
#include "mbtile_ptx.cuh"
#include "mbtile_tcgen05.cuh"

namespace mbt {
namespace {

constexpr int kGradThreads = 256;
constexpr int kGradVecs = 8;                          // 16-byte vectors of a thread and chunk
constexpr int kGradChunk = kGradThreads * kGradVecs;  // vectors
constexpr int kGradCtas = 4;                          // per SM
constexpr int kGradFold = 64;                         // chunks that a thread adds in fp32
constexpr int kGradCluster = 8;                       // CTAs that few chunks are dealt to
// Chunks that one cluster takes (us, cluster / grid, fp32: 100 elements 3.0 / 4.1, 50,000 4.0 /
// 5.1, 100,000 4.9 / 5.2, 200,000 6.1 / 4.7).
constexpr int64_t kGradFewChunks = 16;
// A launch's parameters hold at most 32764 bytes; fewer tensors take a smaller table, whose
// launch has less to send.
constexpr int kGradSmallTable = 32;
constexpr int kGradMiddleTable = 256;
constexpr int kGradLargeTable = 1500;

struct GradTensor {
    char *p;
    int64_t n;
};

struct GradArgs {
    int32_t count;
    int32_t last;              // the call's last launch: sums all partials
    int32_t clip;              // a cluster's launch: multiply, too
    int64_t per;               // chunks a CTA
    double *partial;           // of this launch's CTAs; the call's first are `before` earlier
    int64_t before;
    int32_t *ticket, *clear;
    int64_t clear_n;
    const float *grad_scale;
    float *norm, *scale;
    float max_norm, eps;
};

template <int TABLE>
struct GradTable {
    GradArgs a;
    GradTensor t[TABLE];
    uint32_t end[TABLE];       // chunks up to and with tensor k
    uint8_t type[TABLE];
};

// A tensor's aligned vectors, and the elements before and behind them.
struct GradSpan {
    char *vec;
    int64_t vecs;
    int head, tail;            // elements
};

__host__ __device__ inline GradSpan grad_span(char *p, int64_t n, int es) {
    GradSpan s;
    const int64_t off = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / es;
    s.head = static_cast<int>(off < n ? off : n);
    s.vec = p + s.head * es;
    s.vecs = (n - s.head) * es / 16;
    s.tail = static_cast<int>((n - s.head) - s.vecs * (16 / es));
    return s;
}

inline int64_t grad_chunks(const void *p, int64_t n, int es) {
    const GradSpan s = grad_span(static_cast<char *>(const_cast<void *>(p)), n, es);
    return s.vecs > kGradChunk ? (s.vecs + kGradChunk - 1) / kGradChunk : 1;
}

template <int DT>
__device__ __forceinline__ float squares(const uint4 &v) {
    constexpr int V = Elem<DT>::kVec;
    float f[V];
    unpack<DT>(v, f);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < V; e += 2) s[0] += f[e] * f[e], s[1] += f[e + 1] * f[e + 1];
    return s[0] + s[1];
}

// The sum of a chunk's squares by this thread, in 64 bits (read once more: hardly ever done).
__device__ __noinline__ double wide_squares(const char *vec, int64_t first, int64_t vecs, int type) {
    const int n = type == MBT_F32 ? 4 : 8;
    double sum = 0.0;
#pragma unroll 1
    for (int i = 0; i < kGradVecs; ++i) {
        const int64_t at = first + i * kGradThreads;
#pragma unroll 1
        for (int e = 0; e < n && at < vecs; ++e) {
            const double f = load_any(vec, type, at * n + e);
            sum += f * f;
        }
    }
    return sum;
}

// The sum of a chunk's squares by this thread, and whether any element is not zero.
template <int DT>
__device__ __forceinline__ float chunk_squares(const uint4 (&v)[kGradVecs], bool &any) {
    float s = 0.f;
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < kGradVecs; ++k) {
        s += squares<DT>(v[k]);
        bits |= v[k].x | v[k].y | v[k].z | v[k].w;
    }
    any = (bits & (DT == MBT_F32 ? 0x7fffffffu : 0x7fff7fffu)) != 0;
    return s;
}

// The tensor of chunk c, from tensor k on (end[k - 1] <= c).
template <int TABLE>
__device__ __forceinline__ int grad_find(const GradTable<TABLE> &g, uint32_t c, int k) {
    int lo = k, hi = g.a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (g.end[mid] > c)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// The sum over the CTA, in its first warp.
__device__ __forceinline__ double block_sum(double v, double *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x >= 32) return 0.0;
    v = red[threadIdx.x & (kGradThreads / 32 - 1)];
#pragma unroll
    for (int o = kGradThreads / 64; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The norm and the factor from the sum of all squares; write: to memory, too.
__device__ __forceinline__ float grad_finish(const GradArgs &a, double sum, float gs, bool write) {
    const float norm = static_cast<float>(sqrt(sum) * fabs(static_cast<double>(gs)));
    const float clip = isinf(a.max_norm) ? 1.f : __fdiv_rn(a.max_norm, norm + a.eps);
    const float by = clip >= 1.f ? gs : gs * clip;     // (a NaN norm gives a NaN factor)
    if (write) {
        *a.norm = norm;
        if (a.scale) *a.scale = by;
    }
    return by;
}

template <int DT>
__device__ __forceinline__ uint4 times(const uint4 &v, float by) {
    float f[Elem<DT>::kVec];
    unpack<DT>(v, f);
#pragma unroll
    for (int e = 0; e < Elem<DT>::kVec; ++e) f[e] *= by;
    return pack<DT>(f);
}

// A chunk times a factor.
struct GradChunk {
    GradSpan s;
    char *p;
    int64_t n, chunk, first;
    int type;
    template <int TABLE>
    __device__ __forceinline__ GradChunk(const GradTable<TABLE> &g, int k, int64_t c) {
        type = g.type[k], p = g.t[k].p, n = g.t[k].n;
        s = grad_span(p, n, type == MBT_F32 ? 4 : 2);
        chunk = c - (k ? g.end[k - 1] : 0u);
        first = chunk * kGradChunk + threadIdx.x;
    }
    // (not a read-only load: the vectors are written later)
    __device__ __forceinline__ void load(uint4 (&v)[kGradVecs]) const {
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            const int64_t at = first + i * kGradThreads;
            v[i] = at < s.vecs ? reinterpret_cast<const uint4 *>(s.vec)[at] : make_uint4(0u, 0u, 0u, 0u);
        }
    }
    // This thread's element before or behind the vectors, with the first chunk; -1: none.
    __device__ __forceinline__ int64_t edge() const {
        const int i = threadIdx.x;
        if (chunk != 0 || i >= s.head + s.tail) return -1;
        return i < s.head ? i : n - s.tail + i - s.head;
    }
    __device__ __forceinline__ void scale(const uint4 (&v)[kGradVecs], float by) const {
#pragma unroll
        for (int i = 0; i < kGradVecs; ++i) {
            const int64_t at = first + i * kGradThreads;
            if (at >= s.vecs) continue;
            reinterpret_cast<uint4 *>(s.vec)[at] = type == MBT_F32    ? times<MBT_F32>(v[i], by)
                                                   : type == MBT_BF16 ? times<MBT_BF16>(v[i], by)
                                                                      : times<MBT_F16>(v[i], by);
        }
        const int64_t at = edge();
        if (at >= 0) store_any(p, type, at, load_any(p, type, at) * by);
    }
};

// CLUSTER: a grid of one cluster, whose first CTA adds up the others' sums: a call of few
// chunks waits for no tickets and no memory but its gradients'.
template <int TABLE, bool CLUSTER>
__global__ void __launch_bounds__(kGradThreads, kGradCtas)
    mbt_grad_norm_kernel(const __grid_constant__ GradTable<TABLE> g) {
    __shared__ double red[kGradThreads / 32];
    __shared__ double parts[kGradCluster];
    __shared__ int is_last;
    if constexpr (CLUSTER) cluster_arrive();           // this CTA is there
    const GradArgs &a = g.a;
    const uint32_t chunks = a.count ? g.end[a.count - 1] : 0;
    const int64_t c0 = blockIdx.x * a.per, c1 = min(c0 + a.per, static_cast<int64_t>(chunks));
    float sum = 0.f;
    double wide = 0.0;
    int k = c0 < c1 ? grad_find<TABLE>(g, static_cast<uint32_t>(c0), 0) : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int64_t c = c0; c < c1; ++c) {
        while (g.end[k] <= c) ++k;
        const GradChunk at(g, k, c);
        uint4 v[kGradVecs];
        at.load(v);
        if ((c - c0) % kGradFold == 0) wide += static_cast<double>(sum), sum = 0.f;
        const int type = at.type;
        bool any;
        const float sq = type == MBT_F32    ? chunk_squares<MBT_F32>(v, any)
                         : type == MBT_BF16 ? chunk_squares<MBT_BF16>(v, any)
                                            : chunk_squares<MBT_F16>(v, any);
        if (sq > 0x1p-100f && sq < 0x1p100f)
            sum += sq;
        else if (any)
            wide += wide_squares(at.s.vec, at.first, at.s.vecs, type);
        const int64_t edge = at.edge();
        if (edge >= 0) {
            const float f = load_any(at.p, type, edge);
            wide += static_cast<double>(f) * f;
        }
    }
    const double mine = block_sum(wide + static_cast<double>(sum), red);
    const float gs = a.grad_scale ? *a.grad_scale : 1.f;
    if constexpr (CLUSTER) {
        // every CTA gets all sums (the factor may be written where grad_scale was read)
        cluster_wait();
        if (threadIdx.x < kGradCluster) {
            const double sent = __shfl_sync((1u << kGradCluster) - 1, mine, 0);
            asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(cluster_address(smem_u32(&parts[blockIdx.x]), threadIdx.x)),
                         "d"(sent)
                         : "memory");
        }
        __syncwarp();
        cluster_sync();
        double all = parts[threadIdx.x & (kGradCluster - 1)];
#pragma unroll
        for (int o = kGradCluster / 2; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        const float by = grad_finish(a, all, gs, blockIdx.x == 0 && threadIdx.x == 0);
        if (!a.clip) return;
        for (int64_t c = c1 - 1; c >= c0; --c) {
            while (k > 0 && g.end[k - 1] > c) --k;
            const GradChunk at(g, k, c);
            uint4 v[kGradVecs];
            at.load(v);
            at.scale(v, by);
        }
        return;
    }
    if (threadIdx.x == 0) a.partial[blockIdx.x] = mine;
    if (!a.last) return;
    // the library's other set of tickets is cleared for the next call
    if (blockIdx.x == 0)
        for (int64_t i = threadIdx.x; i < a.clear_n; i += kGradThreads) a.clear[i] = 0;
    if (threadIdx.x == 0) {
        __threadfence();
        is_last = atomicAdd(a.ticket, 1) == static_cast<int>(gridDim.x) - 1;
        __threadfence();
    }
    __syncthreads();
    if (!is_last) return;
    double all = 0.0;
    const double *from = a.partial - a.before;
    for (int64_t i = threadIdx.x; i < a.before + gridDim.x; i += kGradThreads) all += __ldcg(from + i);
    all = block_sum(all, red);
    if (threadIdx.x != 0) return;
    *a.ticket = 0;             // for a replay of this launch
    grad_finish(a, all, gs, true);
}

// A chunk a CTA, whose loads are all under way before the first is used.  (By a grid of
// whole CTAs per SM, as the norm's: bf16 300 M elements 198 us, 6.1 TB/s.)  From the end on:
// what the norm's kernel has read last is still in L2.
template <int TABLE>
__global__ void __launch_bounds__(kGradThreads) mbt_grad_scale_kernel(const __grid_constant__ GradTable<TABLE> g) {
    const GradArgs &a = g.a;
    const uint32_t c = gridDim.x - 1 - blockIdx.x;
    const int k = grad_find<TABLE>(g, c, 0);
    const GradChunk at(g, k, c);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    uint4 v[kGradVecs];
    at.load(v);
    at.scale(v, *a.scale);
}

int es_of(int dtype) { return dtype == MBT_F32 ? 4 : 2; }

int check_grads(const mbt_grad *grads, int64_t count) {
    if (count < 0 || (count > 0 && grads == nullptr)) return MBT_ERR_ARG;
    for (int64_t k = 0; k < count; ++k) {
        const mbt_grad &t = grads[k];
        if (t.n < 0 || t.n > (int64_t{1} << 40) || t.dtype < MBT_F16 || t.dtype > MBT_F32) return MBT_ERR_ARG;
        if (t.n == 0) continue;
        if (!t.grad) return MBT_ERR_ARG;
        if (reinterpret_cast<uintptr_t>(t.grad) % static_cast<uintptr_t>(es_of(t.dtype)) != 0) return MBT_ERR_ALIGN;
    }
    return MBT_OK;
}

// Whether no two tensors share a byte, and none of them any of the scalars.
bool apart(const mbt_grad *grads, int64_t count, std::initializer_list<const float *> scalars, bool *known) {
    struct Range {
        uintptr_t from, to;
    };
    const std::unique_ptr<Range[]> r(new (std::nothrow) Range[static_cast<size_t>(count) + scalars.size()]);
    *known = r != nullptr;
    if (!r) return false;
    int64_t n = 0;
    for (int64_t k = 0; k < count; ++k) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(grads[k].grad);
        if (grads[k].n > 0) r[n++] = {p, p + static_cast<uintptr_t>(grads[k].n * es_of(grads[k].dtype))};
    }
    for (const float *f : scalars) r[n++] = {reinterpret_cast<uintptr_t>(f), reinterpret_cast<uintptr_t>(f + 1)};
    std::sort(r.get(), r.get() + n, [](const Range &x, const Range &y) { return x.from < y.from; });
    for (int64_t k = 1; k < n; ++k)
        if (r[k].from < r[k - 1].to) return false;
    return true;
}

// Fills the table with tensors from *k on; chunks in it.
template <int TABLE>
int64_t fill_table(const mbt_grad *grads, int64_t count, int64_t *k, GradTable<TABLE> *g) {
    int64_t chunks = 0;
    int n = 0;
    for (; *k < count && n < TABLE; ++*k) {
        const mbt_grad &t = grads[*k];
        if (t.n == 0) continue;
        const int64_t c = grad_chunks(t.grad, t.n, es_of(t.dtype));
        if (chunks + c > 0x7fffffff) break;
        chunks += c;
        g->t[n] = {static_cast<char *>(t.grad), t.n};
        g->end[n] = static_cast<uint32_t>(chunks);
        g->type[n] = static_cast<uint8_t>(t.dtype);
        ++n;
    }
    g->a.count = n;
    return chunks;
}

// CTAs and chunks of each.
int grid_of(int64_t chunks, int64_t ctas, int64_t *per) {
    *per = std::max<int64_t>(1, (chunks + ctas - 1) / ctas);
    return static_cast<int>(std::max<int64_t>(1, (chunks + *per - 1) / *per));
}

template <int TABLE>
int run_norm(const mbt_grad *grads, int64_t count, GradArgs a, int sms, cudaStream_t s, bool *clipped) {
    GradTable<TABLE> g;
    if constexpr (TABLE == kGradSmallTable) {
        int64_t k = 0;
        const int64_t chunks = fill_table(grads, count, &k, &g);
        if (chunks <= kGradFewChunks) {
            a.per = (chunks + kGradCluster - 1) / kGradCluster;
            const int32_t filled = g.a.count;
            g.a = a;
            g.a.count = filled;
            *clipped = a.clip != 0;
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(kGradCluster);
            cfg.blockDim = dim3(kGradThreads);
            cfg.stream = s;
            cudaLaunchAttribute attr[2];
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            attr[1].id = cudaLaunchAttributeClusterDimension;
            attr[1].val.clusterDim.x = kGradCluster;
            attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 2;
            return cudaLaunchKernelEx(&cfg, mbt_grad_norm_kernel<TABLE, true>, g) == cudaSuccess ? MBT_OK : MBT_ERR_CUDA;
        }
    }
    // launches of the call, and its CTAs in all
    int64_t launches = 0, ctas = 0;
    for (int64_t k = 0; k < count || launches == 0; ++launches) ctas += grid_of(fill_table(grads, count, &k, &g), kGradCtas * sms, &a.per);
    WorkspaceHold hold;
    int rc = hold.take(s, 1, static_cast<size_t>(ctas) * 8);
    if (rc != MBT_OK) return rc;
    float *partial = nullptr;
    hold.sums(&a.ticket, &a.clear, &a.clear_n, &partial);
    double *const all = reinterpret_cast<double *>(partial);
    int64_t k = 0;
    for (int64_t l = 0; l < launches; ++l) {
        g.a = a;
        g.a.partial = all + a.before;
        g.a.last = l + 1 == launches;
        const int grid = grid_of(fill_table(grads, count, &k, &g), kGradCtas * sms, &g.a.per);
        if (launch_grid(mbt_grad_norm_kernel<TABLE, false>, dim3(static_cast<unsigned>(grid)), kGradThreads, s, g) != cudaSuccess)
            return MBT_ERR_CUDA;
        a.before += grid;
    }
    return MBT_OK;
}

template <int TABLE>
int run_scale(const mbt_grad *grads, int64_t count, const GradArgs &a, cudaStream_t s) {
    GradTable<TABLE> g;
    g.a = a;
    for (int64_t k = 0; k < count;) {
        const int64_t chunks = fill_table(grads, count, &k, &g);
        if (chunks == 0) break;
        if (launch_grid(mbt_grad_scale_kernel<TABLE>, dim3(static_cast<unsigned>(chunks)), kGradThreads, s, g) != cudaSuccess)
            return MBT_ERR_CUDA;
    }
    return MBT_OK;
}

}  // namespace
}  // namespace mbt

namespace mbt {
namespace {

int scale_all(const mbt_grad *grads, int64_t count, const float *scale, cudaStream_t s) {
    GradArgs a{};
    a.scale = const_cast<float *>(scale);
    return count <= kGradSmallTable    ? run_scale<kGradSmallTable>(grads, count, a, s)
           : count <= kGradMiddleTable ? run_scale<kGradMiddleTable>(grads, count, a, s)
                                       : run_scale<kGradLargeTable>(grads, count, a, s);
}

int norm_all(const mbt_grad *grads, int64_t count, const float *grad_scale, float max_norm, float eps, float *norm,
             float *scale, bool clip, cudaStream_t s) {
    int rc = check_grads(grads, count);
    if (rc != MBT_OK) return rc;
    if (!norm || (clip && !scale) || !(max_norm >= 0.f) || !(eps >= 0.f)) return MBT_ERR_ARG;
    for (const void *p : {static_cast<const void *>(grad_scale), static_cast<const void *>(norm), static_cast<const void *>(scale)})
        if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return MBT_ERR_ALIGN;
    bool known = false;
    if (clip && !apart(grads, count, {norm, scale}, &known)) return known ? MBT_ERR_ARG : MBT_ERR_CUDA;
    int sms = 0, optin = 0;
    rc = device_limits(&sms, &optin);
    if (rc != MBT_OK) return rc;
    GradArgs a{};
    a.grad_scale = grad_scale;
    a.norm = norm;
    a.scale = scale;
    a.max_norm = max_norm;
    a.eps = eps;
    a.clip = clip;
    bool clipped = false;
    rc = count <= kGradSmallTable    ? run_norm<kGradSmallTable>(grads, count, a, sms, s, &clipped)
         : count <= kGradMiddleTable ? run_norm<kGradMiddleTable>(grads, count, a, sms, s, &clipped)
                                     : run_norm<kGradLargeTable>(grads, count, a, sms, s, &clipped);
    return rc == MBT_OK && clip && !clipped ? scale_all(grads, count, scale, s) : rc;
}

}  // namespace
}  // namespace mbt

extern "C" int tile_grad_norm(const mbt_grad *grads, int64_t count, const float *grad_scale, float max_norm, float eps,
                              float *norm, float *scale, void *stream) {
    return mbt::norm_all(grads, count, grad_scale, max_norm, eps, norm, scale, false, static_cast<cudaStream_t>(stream));
}

extern "C" int tile_grad_clip(const mbt_grad *grads, int64_t count, const float *grad_scale, float max_norm, float eps,
                              float *norm, float *scale, void *stream) {
    return mbt::norm_all(grads, count, grad_scale, max_norm, eps, norm, scale, true, static_cast<cudaStream_t>(stream));
}

extern "C" int tile_grad_scale(const mbt_grad *grads, int64_t count, const float *scale, void *stream) {
    using namespace mbt;
    const int rc = check_grads(grads, count);
    if (rc != MBT_OK) return rc;
    if (count == 0) return MBT_OK;
    if (!scale) return MBT_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(scale) % 4 != 0) return MBT_ERR_ALIGN;
    bool known = false;
    if (!apart(grads, count, {scale}, &known)) return known ? MBT_ERR_ARG : MBT_ERR_CUDA;
    return scale_all(grads, count, scale, static_cast<cudaStream_t>(stream));
}
