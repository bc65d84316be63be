// Device and host helpers of the 8-bit floating-point products (sm_103a): hand-overs across clusters
// and pairs of CTAs, tensor memory, tensor maps.
#pragma once

// poll without sleeping: the waits are short and on the critical path
#ifndef H32_WAIT_SLEEP
#define H32_WAIT_SLEEP 0
#endif

#include "h32_common.cuh"
#include "h32_tmap.cuh"

#include <cuda_bf16.h>

#include <atomic>

namespace h32 {
namespace {

constexpr int kMaxExperts = 1024;

// 32 lanes x 32 bit, 32 consecutive columns per thread
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// wait for the loads issued; `r`, one of them, is read after it
__device__ __forceinline__ void tmem_wait_for(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29])
                 :);
    asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}


// clusters -------------------------------------------------------------------
__device__ __forceinline__ void peer_store(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// arrive on another CTA's barrier, handing over what the warp stored
__device__ __forceinline__ void peer_arrive_release(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// wait (bounded, warp-uniform outcome) for arrivals that release other CTAs' writes
__device__ __forceinline__ bool warp_wait_cluster(uint64_t *bar, uint32_t parity, uint64_t limit,
                                                  volatile int *abort) {
    bool ok = false;
    for (uint64_t i = 0; i < limit && !ok; ++i) {
        uint32_t r;
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
            "selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(r)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        ok = r != 0;
        if (!ok && *abort) break;
    }
    return __all_sync(0xFFFFFFFFu, ok);
}
// the same for what other CTAs release, as warp_wait_or_look
__device__ __forceinline__ bool warp_wait_or_look_cluster(uint64_t *bar, uint32_t parity, uint64_t limit,
                                                          volatile int *abort) {
    uint32_t all;
    asm volatile(
        "{\n.reg .pred p, q;\nmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        "vote.sync.all.pred q, p, 0xffffffff;\nselp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(all)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (all) return true;
    if (limit == 1) return false;
    return warp_wait_cluster(bar, parity, limit, abort);
}
// Arrive on another CTA's barrier, handing over tensor memory that this warp has read: its loads
// were waited for (tcgen05.wait::ld) and fenced (tcgen05.fence::before_thread_sync), and the
// issuer of the products that overwrite it fences behind its wait.  That pattern orders tensor
// memory with relaxed arrivals; nothing else may rest on this one.  (A release, which waits for
// more than the thread's own accesses, doubled the time of 4096 x 34816 x 5120.)
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// CTA pairs: tensor memory and products of both CTAs (cta_group::2) ------------
// allocation and release: one warp of each CTA of the pair
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst_smem, uint32_t ncols) {
    asm volatile(
        "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n"
        "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(smem_u32(dst_smem)),
        "r"(ncols)
        : "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// a box of a tensor to this CTA's shared memory, complete on a barrier in either CTA of the pair
// (`bar`: its address there)
__device__ __forceinline__ void tma_load_2d_pair(void *smem_dst, const void *tmap, uint32_t bar, int32_t x, int32_t y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}
// counts `bytes` as arrived, without a copy
__device__ __forceinline__ void mbar_complete_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
// the descriptors' addresses hold in both CTAs; one thread of the first one issues
__device__ __forceinline__ void mma_pair_f8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// arrive on the barrier at this place in both CTAs once this thread's products are done
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// Once a kernel and device: its dynamic shared memory may be up to `bytes`.
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
    static std::atomic<uint64_t> done{0};   // a bit a device (check_device admits 64)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (done.load(std::memory_order_relaxed) >> dev & 1)) return e;
    e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return e;
}

// tensor maps ----------------------------------------------------------------
// rows of K code bytes, boxes of `box_rows` rows x 128 bytes, 128B-swizzled; rows and
// columns outside the array read as zero
inline bool code_map(CUtensorMap *map, const void *base, uint64_t K, uint64_t rows, uint32_t box_rows) {
    const cuuint64_t dims[2] = {K, rows}, strides[1] = {K};
    const cuuint32_t box[2] = {128, box_rows}, estr[2] = {1, 1};
    return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// the group-major scales [groups][ld], boxes of `box` scales of one group
inline bool scale_map(CUtensorMap *map, const void *base, uint64_t ld, uint64_t groups, uint32_t box_cols) {
    const cuuint64_t dims[2] = {ld, groups}, strides[1] = {ld * 4};
    const cuuint32_t box[2] = {box_cols, 1}, estr[2] = {1, 1};
    return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace h32
