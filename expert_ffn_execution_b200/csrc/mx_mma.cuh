// mx_mma.cuh -- the sm_100a block-scaled tensor-core instructions: scales
// from shared into tensor memory, tcgen05.mma of MXFP4 x MXFP4 (kind::mxf4,
// K = 64 an instruction) and of E4M3 / E2M1 operands (kind::mxf8f6f4, K = 32).
#pragma once

#include "mx.cuh"
#include "tc05.cuh"

namespace strata {

// Descriptor words of one 512-byte scale tile in shared memory: unswizzled,
// 32 rows of 16 bytes, 8-row groups 128 bytes apart, version 1.
STRATA_DEVFN uint32_t smem_desc_scale_lo(uint32_t saddr) {
  return ((saddr >> 4) & 0x3FFFu) | (1u << 16);
}
constexpr uint32_t kScaleDescHi = (128u >> 4) | (1u << 14);

// Copies one scale tile into four tensor-memory columns at taddr, the 32
// lanes repeated in all four lane quarters: column c, lane l then holds row
// 32 c + l's four scale bytes.
STRATA_DEVFN void tmem_cp_scales(uint32_t taddr, uint32_t desc_lo) {
  asm volatile(
      "{\n\t.reg .b64 sd;\n\t"
      "mov.b64 sd, {%1, %2};\n\t"
      "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], sd;\n\t}" ::"r"(taddr),
      "r"(desc_lo), "r"(kScaleDescHi)
      : "memory");
}

// Instruction descriptor: both operands K-major, E8M0 scales, M = m, N = n.
// afmt / bfmt: kind::mxf8f6f4 counts E4M3 as 0 and E2M1 as 5, kind::mxf4
// E2M1 as 1.  sf: which byte of the 32-bit scale columns the instruction's
// (first) scale is.
__host__ __device__ constexpr uint32_t idesc_mx(uint32_t afmt, uint32_t bfmt, int m, int n,
                                                 uint32_t sf) {
  return (sf << 4) | (afmt << 7) | (bfmt << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         ((uint32_t)(m >> 7) << 27) | (sf << 29);
}

template <bool F4>
STRATA_DEVFN void mma_mx(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                         uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (F4) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.b32 p, %7, 0;\n\t"
        "mov.b64 ad, {%1, %3};\n\t"
        "mov.b64 bd, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], ad, bd, %4, [%5], "
        "[%6], p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.b32 p, %7, 0;\n\t"
        "mov.b64 ad, {%1, %3};\n\t"
        "mov.b64 bd, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], ad, bd, %4, "
        "[%5], [%6], p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  }
}

// ---------------------------------------------------------------- CTA pairs
// The same instructions over a pair of CTAs (cta_group::2, issued by the even
// CTA): A is 128 rows of each CTA, B half of its N rows in each CTA, D 128
// lanes x N columns in each; the copies run in both, from each CTA's own
// shared memory to its own tensor memory.
STRATA_DEVFN void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst_smem)),
               "r"(ncols)
               : "memory");
}
STRATA_DEVFN void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
STRATA_DEVFN void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
STRATA_DEVFN void tmem_cp_scales_pair(uint32_t taddr, uint32_t desc_lo) {
  asm volatile(
      "{\n\t.reg .b64 sd;\n\t"
      "mov.b64 sd, {%1, %2};\n\t"
      "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], sd;\n\t}" ::"r"(taddr),
      "r"(desc_lo), "r"(kScaleDescHi)
      : "memory");
}
template <bool F4>
STRATA_DEVFN void mma_mx_pair(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                              uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (F4) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.b32 p, %7, 0;\n\t"
        "mov.b64 ad, {%1, %3};\n\t"
        "mov.b64 bd, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], ad, bd, %4, [%5], "
        "[%6], p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
        "setp.ne.b32 p, %7, 0;\n\t"
        "mov.b64 ad, {%1, %3};\n\t"
        "mov.b64 bd, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], ad, bd, %4, "
        "[%5], [%6], p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  }
}
// Arrive on the barrier at `bar`'s offset in both CTAs once the tcgen05
// operations this thread has issued are complete.
STRATA_DEVFN void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// 2-D tiled load into this CTA's shared memory that counts its bytes on a
// barrier of either CTA of the pair (`bar`: its shared::cluster address).
STRATA_DEVFN void tma_load_2d_pair(void* dst, const CUtensorMap* map, int c0, int c1,
                                   uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
// 32 lanes x 32 bits, 32 consecutive columns a thread.
STRATA_DEVFN void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// ---------------------------------------------------------------- clusters
// The shared::cluster address of `saddr`'s offset in CTA `rank` of the cluster.
STRATA_DEVFN uint32_t cluster_addr(uint32_t saddr, uint32_t rank) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(saddr), "r"(rank));
  return ra;
}
// Arrive on another CTA's barrier.  For hand-overs that order tensor memory
// (by its own fences), not ordinary memory: a release at cluster scope would
// wait a thousand cycles and more for the thread's global writes.
STRATA_DEVFN void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The cluster's barrier, in two steps, without ordering memory: for mbarriers
// made visible by their own fence, and for shared memory that only has to stay allocated.
// (A release waits for the CTA's outstanding global writes: 0.5 us and more.)
STRATA_DEVFN void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
STRATA_DEVFN void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
STRATA_DEVFN void cluster_sync_relaxed() {
  cluster_arrive_relaxed();
  cluster_wait();
}
STRATA_DEVFN uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Bulk copy of this CTA's shared memory into another's (`dst`, `bar`: their
// shared::cluster addresses), counted in bytes on that CTA's barrier.
STRATA_DEVFN void bulk_s2cluster(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, "
      "[%3];" ::"r"(dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}

}  // namespace strata
