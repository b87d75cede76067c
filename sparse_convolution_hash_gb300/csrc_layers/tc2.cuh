// tc2.cuh -- inline-PTX wrappers beyond csrc/ptx.cuh: thread-block clusters, TMA
// loads of 2-D and 3-D tiles, and the tensor-core operations in their
// one-CTA (CG = 1) and CTA-pair (CG = 2) forms.
#pragma once

#include "ptx.cuh"

namespace spc {
namespace ptx {

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address, in the cluster's shared window, of a shared variable of CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}

// Arrives on another CTA's mbarrier.  Nothing written by this thread crosses over with it (what
// the barrier hands over is a stage of this CTA's own shared memory, or tensor memory), so it orders this
// CTA's accesses only: at cluster scope each arrival waited about a microsecond for them.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// TMA loads that complete on an mbarrier named by its cluster address (for a
// CTA pair, the leader's).
template <int CG>
__device__ __forceinline__ void tma_load2d(uint32_t dst, const void* tmap, int32_t x, int32_t y, uint32_t bar)
{
    if constexpr (CG == 1)
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
                     " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(bar)
                     : "memory");
}

template <int CG>
__device__ __forceinline__ void tma_load3d(uint32_t dst, const void* tmap, int32_t x, int32_t y, int32_t z,
                                           uint32_t bar)
{
    if constexpr (CG == 1)
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
                     " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar)
                     : "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_alloc_cg(uint32_t* dst_smem, uint32_t ncols)
{
    if constexpr (CG == 1) {
        tmem_alloc(dst_smem, ncols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
                     "tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::"r"(smem_u32(dst_smem)),
                     "r"(ncols)
                     : "memory");
    }
}

template <int CG>
__device__ __forceinline__ void tmem_dealloc_cg(uint32_t taddr, uint32_t ncols)
{
    if constexpr (CG == 1)
        tmem_dealloc(taddr, ncols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// D[tmem] (+)= A B, 16-bit operands in shared memory, K = 16; for a pair M spans both CTAs
// and each holds half of B's columns.
template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate)
{
    if constexpr (CG == 1)
        mma<0>(tmem_d, adesc, bdesc, idesc, accumulate);
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "setp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
                     "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
                     : "memory");
}

// Arrives, in every CTA of the pair, on the mbarrier at this offset once the
// MMAs issued so far by this thread have completed.
template <int CG>
__device__ __forceinline__ void mma_commit_cg(uint64_t* bar)
{
    if constexpr (CG == 1)
        mma_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
                     " [%0], %1;" ::"r"(smem_u32(bar)), "h"((uint16_t)3)
                     : "memory");
}

}  // namespace ptx
}  // namespace spc
