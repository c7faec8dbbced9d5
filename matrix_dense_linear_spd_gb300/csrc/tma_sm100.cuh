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

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *mbar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];\n" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(mbar)), "r"(x), "r"(y), "r"(z)
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

__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

}  // namespace tc
}  // namespace bl
