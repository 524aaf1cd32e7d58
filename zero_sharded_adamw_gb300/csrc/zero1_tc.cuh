// zero1_tc.cuh -- inline-PTX building blocks of the tensor-core kernels
// (sm_103a): tiled TMA loads, tcgen05 matrix products with accumulators in
// tensor memory, and the fences between the kernel's roles.
#pragma once

#include <cuda.h>   // CUtensorMap
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "zero1_ptx.cuh"

namespace zero1 {
namespace tc {

using ptx::smem_u32;

// ------------------------------------------------------------ tiled TMA

// Box of a 3-D tensor map (x fastest) into shared memory of this block of a
// pair; its bytes are counted on a barrier of either block, given by its
// cluster address.  x times the element size is a multiple of 16 bytes.
__device__ __forceinline__ void tma_box_pair(uint32_t smem_dst, const CUtensorMap *map, int x, int y, int z,
                                             uint32_t cluster_bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3, %4}], [%5];" ::"r"(smem_dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(cluster_bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Order generic-proxy accesses of global memory before later async-proxy
// (TMA) accesses, and the other way round.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// ------------------------------------------------------------ cross-CTA flags

__device__ __forceinline__ unsigned ld_acquire(const unsigned *p)
{
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void red_release_add(unsigned *p, unsigned v)
{
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// ------------------------------------------------------------ block pairs

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Cluster address of the same shared-memory place in block `rank` of the pair.
__device__ __forceinline__ uint32_t map_to(uint32_t smem_addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

// The same without ordering this thread's writes before it (which would wait
// for its stores to global memory).
__device__ __forceinline__ void arrive_cluster_relaxed(uint32_t cluster_bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}

__device__ __forceinline__ void st_cluster(uint32_t cluster_addr, uint4 v)
{
    asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

// ptx::mbar_test with acquire at cluster scope: what either block of the
// pair wrote before it arrived is visible after it.
__device__ __forceinline__ bool pair_test(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{ .reg .pred q; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 q, [%1], %2; selp.u32 %0, 1, 0, q; }"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// The same without waiting at all (try_wait above may suspend the thread for
// some microseconds before it answers no).
__device__ __forceinline__ bool pair_peek(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{ .reg .pred q; mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 q, [%1], %2; selp.u32 %0, 1, 0, q; }"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// ptx::mbar_wait's limits and error reporting, over pair_test.
__device__ __forceinline__ bool pair_wait(uint64_t *bar, uint32_t parity, volatile int *abort, unsigned *errors)
{
    if (pair_test(bar, parity)) return true;
    const unsigned long long t0 = ptx::global_ns();
    for (uint32_t i = 1;; ++i) {
        if (pair_test(bar, parity)) return true;
        if ((i & 63u) == 0) {
            if (*abort) return false;
            if (ptx::global_ns() - t0 > ptx::kWaitLimitNs) {
                *abort = 1;
                atomicOr(errors, kErrWaitTimeout);
                return false;
            }
        }
    }
}

// ------------------------------------------------------------ tcgen05

// The products span a pair of blocks on neighbouring SMs (cta_group::2): one
// thread of the first block issues them, each block holds its half of A, of
// B and of the accumulators.

// Allocate `cols` (a power of two, at least 32) TMEM columns in both blocks;
// one converged warp of each.  The base address is written to *smem_slot.
__device__ __forceinline__ void tmem_alloc(uint32_t *smem_slot, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D[tmem] (+)= A * B, f16 operands in shared memory, fp32 accumulators.
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// One arrival on `bar` of both blocks when every product issued so far by
// this thread is done.
__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// 32 lanes (this warp's quarter) x 16 fp32 columns of TMEM, one row a lane.
__device__ __forceinline__ void tmem_load16(float v[16], uint32_t addr)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(v);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}

// ------------------------------------------------------------ shared memory

__device__ __forceinline__ uint4 ld_shared(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ void st_shared(uint32_t addr, uint4 v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint16_t v)
{
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// The same for one block by itself (cta_group::1).
__device__ __forceinline__ void tmem_alloc1(uint32_t *smem_slot, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_slot)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free1(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void mma1_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}
__device__ __forceinline__ void mma1_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle, tiles made of boxes of
// 64 f16 (128 bytes) by 64 or 128 rows, `box` bytes each:
//   K-major:  the box's rows are M (or N) and its columns K; 8-row groups
//             follow at 1024 bytes (SBO), K within one box (LBO unused);
//   MN-major: the box's rows are K and its columns M (or N); 8-row groups of
//             K follow at 1024 bytes (SBO), the next 64 of M (or N) one box
//             further (LBO).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, bool mn_major, uint32_t box = 8192)
{
    const uint64_t lbo = mn_major ? (box >> 4) : 1u;
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (lbo << 16) | ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// Descriptor step for 16 further K: 32 bytes along a K-major row, 16 rows of
// 128 bytes in an MN-major box.
__device__ __forceinline__ uint64_t k16_step(bool mn_major) { return mn_major ? (2048u >> 4) : (32u >> 4); }

// Instruction descriptor: f16 x f16 -> fp32, M x N, operands K- or MN-major.
__device__ __forceinline__ uint32_t instr_desc(uint32_t m, uint32_t n, bool a_mn, bool b_mn)
{
    return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

}  // namespace tc
}  // namespace zero1
