// tcgen05 and TMA wrappers of the 8-bit operators (sm100.cuh has the rest): the block-scaled 8-bit
// MMA, CTA pairs (cta_group::2) and narrow TMEM loads.
//
// The issuing functions are called by a whole, converged warp and take a flag that is set in one
// of its lanes (elect_one): their operands then live in uniform registers. Called from a branch
// of one lane they are moved there for every instruction, which made an MMA loop of 4
// instructions and a commit cost 600 cycles a round.
#pragma once
#include "sm100.cuh"

namespace kq {

__device__ __forceinline__ uint32_t elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e;
}
// A warp index that the compiler knows to be the same in all lanes.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0); }

__device__ __forceinline__ void expect_tx_if(uint32_t on, uint32_t bar, uint32_t bytes) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
               "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}"
               ::"r"(bar), "r"(bytes), "r"(on) : "memory");
}
// 2-D tiled load (no multicast) into this CTA's shared memory.
__device__ __forceinline__ void tma_load_if(uint32_t on, uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y,
                                            uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar), "r"(on) : "memory");
}
// The same, completing on a barrier of either CTA of a pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_pair_if(uint32_t on, uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y,
                                                 uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3}], [%4];\n\t}"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar), "r"(on) : "memory");
}
// Plain bulk copy, 16-byte aligned addresses and size.
__device__ __forceinline__ void bulk_load_if(uint32_t on, uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
      "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "r"(on) : "memory");
}

// D(tmem) (+)= (A * 2^sfa)(smem) * (B * 2^sfb)(smem)^T, 8-bit inputs (E4M3 per idesc), K = 32
// per instruction with one E8M0 scale per row (scales read from TMEM). PAIR: one MMA over both
// CTAs' operands and accumulators (M = 256).
template <bool PAIR>
__device__ __forceinline__ void mma_mxf8_if(uint32_t on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(on) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb), "r"(on) : "memory");
}
// A 512-byte scale atom to 4 TMEM columns, replicated to the four lane quadrants (PAIR: each
// CTA's shared memory to its own TMEM).
template <bool PAIR>
__device__ __forceinline__ void scale_cp_if(uint32_t on, uint32_t taddr, uint64_t sdesc) {
  if (PAIR)
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}"
                 ::"r"(taddr), "l"(sdesc), "r"(on) : "memory");
  else
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}"
                 ::"r"(taddr), "l"(sdesc), "r"(on) : "memory");
}
// Arrive on a barrier (PAIR: on the one at this address in the cluster's CTAs `ctas`, a bit each)
// when the tcgen05 work that the electing lane issued so far is done.
template <bool PAIR>
__device__ __forceinline__ void commit_if(uint32_t on, uint32_t bar, uint16_t ctas = 0) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}"
        ::"r"(bar), "h"(ctas), "r"(on) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(bar), "r"(on) : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* smem_slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
               ::"r"(smem_u32(smem_slot)), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// Arrive on a barrier of any CTA of the cluster (a shared::cluster address). Relaxed, since it passes on
// TMEM columns and no memory: the loads from them have ended (tcgen05.wait::ld), and the fences
// tcgen05.fence::before_thread_sync ahead of it and ::after_thread_sync behind the wait order them
// before the MMAs that follow there, which is what the PTX ISA asks of tcgen05 operations of
// different threads. A release would wait for this thread's stores to global memory too.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The two halves of cluster_sync.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_shared_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// mbar_wait for a barrier on which other CTAs of the cluster arrive.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, uint32_t* err,
                                                  uint32_t code, uint64_t limit_ns) {
  const uint32_t a = smem_u32(bar);
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(a), "r"(parity) : "memory");
    if (ok) return true;
    if (i == 0) t0 = globaltimer_ns();
    else if ((i & 255u) == 0u && globaltimer_ns() - t0 > limit_ns) {
      if (err) atomicOr(err, code);
      return false;
    }
  }
}

// drain_ring for an MMA issuer whose wait ran out after `taken` of `total` k-tiles: waits, limit_ns at
// most for each slot and without reporting, for the loads that are under way or about to be (a
// producer is a ring ahead), since no copy may still land when the CTA goes on.
__device__ __forceinline__ void drain_after(uint64_t* full, int stages, int64_t taken, int64_t total, uint64_t limit_ns) {
  for (int64_t j = taken; j < min(taken + stages, total); ++j)
    mbar_wait(&full[j % stages], static_cast<uint32_t>(j / stages) & 1u, nullptr, 0u, limit_ns);
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

// W columns of this thread's TMEM lane from `col` on: added to v where `more`, else v itself.
template <int W>
__device__ __forceinline__ void add_columns(uint32_t col, bool more, float* v) {
#pragma unroll
  for (int c = 0; c < W; c += 16) {
    uint32_t r[16];
    tmem_ld_32x32b_x16(col + c, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[c + i] = __uint_as_float(r[i]) + (more ? v[c + i] : 0.f);
  }
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
