// Tensor copies (TMA) and kind::f16 matrix instructions for sm_103a, in inline PTX: what the
// tiled bf16 products need beside tc_sm100.cuh.
//
// Operand tiles are 64 bf16 values (128 bytes) wide in memory's contiguous direction, written by
// TMA with the 128-byte swizzle: line r of a tile at r*128 bytes, its 16-byte chunk c at
// c XOR (r mod 8). If the contiguous direction is the product's K the tile is "K-major" (a line
// is one row of A or B); if it is M or N the tile is "MN-major" (a line is one k).
#pragma once

#include <cuda.h>

#include "tc_sm100.cuh"

namespace bl {
namespace tc {

// ---- CTA pairs (clusters of two): both CTAs run the same layout of shared memory, and the even
// one, the leader, issues the products of both.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// Shared-memory address, valid in the whole cluster, of the leader's variable at the same place.
__device__ __forceinline__ uint32_t at_leader(const void *p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;\n" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_addr) : "memory");
}

// Global tile -> this CTA's shared memory; `mbar` (a cluster address; with CTAS = 2 it may be the
// leader's) counts the bytes.
template <int CTAS>
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint32_t mbar, int x, int y, int z) {
    if constexpr (CTAS == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
            "[%2];\n" ::"r"(smem_u32(dst)),
            "l"(map), "r"(mbar), "r"(x), "r"(y), "r"(z)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%3, %4, %5}], [%2];\n" ::"r"(smem_u32(dst)),
            "l"(map), "r"(mbar), "r"(x), "r"(y), "r"(z)
            : "memory");
}
// Shared memory -> global tile (add: f32 sums, formed in L2), tracked by bulk groups as in
// bulk_reduce_add_f32. What lies outside the tensor is not written.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int x, int y, int z, bool add) {
    if (add)
        asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n" ::"l"(map),
                     "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];\n" ::"l"(map),
                     "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
                     : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(map) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t *mbar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(mbar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *mbar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(mbar)) : "memory");
}

// Move registers between the block's warpgroups (every warp of a group executes it; the groups'
// shares together must not exceed what the block was launched with).
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}

// Shared-memory matrix descriptor of an MN-major tile: consecutive groups of 8 k lie 1024 bytes
// apart (stride offset), consecutive groups of 64 M or N values `group` bytes apart (leading
// offset); version and swizzle bits as in sdesc_sw128.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t group) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFF) >> 4);
    d |= static_cast<uint64_t>(group >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// Instruction descriptor, kind::f16 with bf16 A and B and an f32 D: bits 15 and 16 mark A and B
// as MN-major, the other fields as in idesc_tf32.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(a_mn) << 15) |
           (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

template <int CTAS>
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate) {
    if constexpr (CTAS == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
            : "memory");
}
// Arrive, in every CTA of the group, on the mbarrier at this place once all products issued so
// far are done.
template <int CTAS>
__device__ __forceinline__ void mma_commit_all(uint64_t *mbar) {
    if constexpr (CTAS == 1) mma_commit(mbar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
                smem_u32(mbar)),
            "h"(static_cast<uint16_t>(3))
            : "memory");
}
template <int CTAS>
__device__ __forceinline__ void tmem_take(uint32_t *slot_smem, uint32_t ncols) {
    if constexpr (CTAS == 1) {
        tmem_alloc(slot_smem, ncols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(slot_smem)), "r"(ncols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
    }
}
template <int CTAS>
__device__ __forceinline__ void tmem_give(uint32_t taddr, uint32_t ncols) {
    if constexpr (CTAS == 1) tmem_dealloc(taddr, ncols);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(ncols) : "memory");
}

}  // namespace tc
}  // namespace bl
