// PTX wrappers, bounded waits and the launch helper that every translation
// unit's kernels share.
#pragma once

#include "internal.h"

namespace mbt {
namespace {

// ---------------------------------------------------------------------------
// PTX wrappers
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count)
                 : "memory");
}

// Make barrier initialisation visible to the copy engine before first use.
__device__ __forceinline__ void fence_barrier_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One probe of the barrier: true once the phase with parity `parity` is over.
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}

__device__ __forceinline__ uint64_t global_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// 1-D bulk copy of `bytes` bytes (16-byte aligned address and size) from
// global memory into shared memory; completion is counted on `bar` in bytes.
__device__ __forceinline__ void bulk_load_1d(uint32_t dst, const void *src, uint32_t bytes,
                                             uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
            dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// Bulk tensor copy of one 2-D box at element coordinates (x = column, y = row)
// into shared memory; completion is counted on `bar` in bytes.
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map,
                                            int32_t x, int32_t y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Bulk tensor copy of one 2-D box from shared memory to global memory at
// element coordinates (x, y); elements outside the tensor are not written.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int32_t x,
                                             int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(src), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void bulk_commit_group() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// Wait until at most one committed bulk store group still reads shared memory.
__device__ __forceinline__ void bulk_wait_read_allow1() {
    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}

__device__ __forceinline__ void bulk_wait_read_all() {
    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

__device__ __forceinline__ void bulk_wait_all() {
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void stg128(void *ptr, const uint4 &v) {
    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(ptr), "r"(v.x),
                 "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

// ---------------------------------------------------------------------------
// Bounded waits and the failure record
// ---------------------------------------------------------------------------
struct WaitCtl {
    uint64_t budget_ns;
    volatile int *abort;
    int32_t *status;    // where a timed-out wait is recorded: the call's own
                        // status buffer (mbt_opts.status) or g_status
};

__device__ bool wait_bounded(uint32_t bar, uint32_t parity, const WaitCtl &w,
                             bool heed_abort) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    // Each probe costs well over 8 ns, so this iteration cap is reached only
    // if the timer itself stalls; it keeps the loop finite regardless.
    const uint64_t max_iter = w.budget_ns / 8 + 4096;
    for (uint64_t it = 0; it < max_iter; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 7) == 7) {
            if (heed_abort && *w.abort) return false;
            if (global_ns() - t0 > w.budget_ns) return false;
        }
    }
    return false;
}

__device__ void report_timeout(const WaitCtl &w, int role, uint32_t stage, uint32_t parity) {
    int32_t *st = w.status;
    if (atomicCAS(&st[0], 0, static_cast<int32_t>(MBT_ERR_TIMEOUT)) == 0) {
        st[1] = static_cast<int32_t>(blockIdx.x);
        st[2] = static_cast<int32_t>(stage);
        st[3] = role * 2 + static_cast<int32_t>(parity);
    }
}

// Launch of a pipeline kernel with programmatic stream serialization: it may be
// launched, and its CTAs set up their shared memory, while the previous kernel
// of the stream completes (a host launch otherwise starts ~3 us after it
// ends); init_pipeline holds every global access until that kernel has
// completed.
template <class... P, class... A>
cudaError_t launch_pipeline(void (*kernel)(P...), int grid, int threads, int smem,
                            cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace
}  // namespace mbt
