// sm100_mma.cuh — what the matrix product uses beside sm100.cuh: 2-D TMA maps
// and loads, 8-bit tcgen05.mma, CTA pairs (cta_group::2), clusters, and the
// bounded wait with its abort mode.
#pragma once

#include <cuda.h>

#include "sm100.cuh"
#include "tma_map.cuh"

namespace ssd {
namespace sm100 {

// ---------------------------------------------------------------- host side

// Map over `rows` rows of `cols` elements, `pitch` bytes apart, read in boxes of
// box_rows x 128 bytes with the 128-byte swizzle; what lies past an extent reads
// as zero. False when the driver refuses the sizes.
inline bool make_map_rows(CUtensorMap* map, const void* base, bool e4m3, uint64_t cols, uint64_t rows,
                          uint64_t pitch, uint32_t box_rows)
{
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch};
    const cuuint32_t box[2] = {e4m3 ? 128u : 64u, box_rows}, estr[2] = {1, 1};
    return enc(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ----------------------------------------------------------------- clusters

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Address of this CTA's shared-memory location in the CTA of the given rank.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float ld_cluster_f1(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// ----------------------------------------------------------------------- TMA

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int c0, int c1, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(smem_addr(bar))
        : "memory");
}

// Brings a box into L2 alone.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int c0, int c1)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1)
                 : "memory");
}

// A load for a CTA pair: the bytes land in this CTA, the barrier (a
// shared::cluster address) may be the pair's other CTA's.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// ------------------------------------------------------------------- tcgen05

// Instruction descriptor of e4m3 operands (kind::f8f6f4), K-major, fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N)
{
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] B[smem]^T, one K step of 32 bytes per row; PAIR: issued
// by the leader for both CTAs, each of which holds half of A's and of B's rows.
template <bool E4M3, bool PAIR>
__device__ __forceinline__ void mma_step(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         bool accumulate)
{
#define SSD_MMA(GROUP, KIND)                                                                            \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma." GROUP ".kind::" KIND    \
                 " [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),                                            \
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u) : "memory")
    if constexpr (PAIR) {
        if constexpr (E4M3) SSD_MMA("cta_group::2", "f8f6f4");
        else SSD_MMA("cta_group::2", "f16");
    } else {
        if constexpr (E4M3) SSD_MMA("cta_group::1", "f8f6f4");
        else SSD_MMA("cta_group::1", "f16");
    }
#undef SSD_MMA
}

// Arrive on the barrier of this offset in both CTAs of the pair once every MMA
// issued so far by this thread has completed.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst_smem)),
                 "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// -------------------------------------------------------------- bounded wait

constexpr uint64_t kPollLimit = 1ull << 22;

// Waits for the phase of the given parity. A wait that gives up records the
// device status and puts the CTA into its abort mode (the flag in shared
// memory), in which every wait returns at once.
__device__ __forceinline__ void wait_or_abort(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                              unsigned int* status)
{
    if (mbar_try_wait_1us(bar, parity)) return;
    for (uint64_t i = 0; i < kPollLimit && !*abort_flag; ++i)
        if (mbar_try_wait_1us(bar, parity)) return;
    *abort_flag = 1;
    if (status) atomicCAS(status, 0u, 1u);  // kDevWaitTimeout
}

}  // namespace sm100
}  // namespace ssd
