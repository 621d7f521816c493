// tcgen05 wrappers of the 8-bit operators (sm100.cuh has the rest): the block-scaled 8-bit MMA
// and narrow TMEM loads.
#pragma once
#include "sm100.cuh"

namespace kq {

// D(tmem) (+)= (A * 2^sfa)(smem) * (B * 2^sfb)(smem)^T, 8-bit inputs (E4M3 per idesc), K = 32
// per instruction with one E8M0 scale per row (scales read from TMEM).
__device__ __forceinline__ void mma_mxf8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem),
        "r"(sfb_tmem)
      : "memory");
}
// Each thread of the warp reads 16 consecutive 32-bit columns of its own TMEM lane.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// kind::mxf8f6f4 (block32): E4M3 A/B, E8M0 scales, K = 32 per instruction, both K-major.
// sf_id selects the byte (0 .. 3) of the 32-bit TMEM scale column of A and of B.
__host__ __device__ constexpr uint32_t idesc_mxf8(uint32_t M, uint32_t N, uint32_t sf_id) {
  return (sf_id << 4)         // B scale-factor byte id
       | (0u << 7)            // A format: E4M3
       | (0u << 10)           // B format: E4M3
       | ((N >> 3) << 17)     // N / 8
       | (1u << 23)           // scale format: E8M0
       | ((M >> 4) << 24)     // M / 16
       | (sf_id << 29);       // A scale-factor byte id
}

}  // namespace kq
