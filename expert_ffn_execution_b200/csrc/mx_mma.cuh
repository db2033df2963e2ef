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

// Instruction descriptor: both operands K-major, E8M0 scales, M = m, N = n.
// afmt / bfmt: kind::mxf8f6f4 counts E4M3 as 0 and E2M1 as 5, kind::mxf4
// E2M1 as 1.  sf: which byte of the 32-bit scale columns the instruction's
// (first) scale is.
__host__ __device__ constexpr uint32_t idesc_mx(uint32_t afmt, uint32_t bfmt, int m, int n,
                                                 uint32_t sf) {
  return (sf << 4) | (afmt << 7) | (bfmt << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         ((uint32_t)(m >> 7) << 27) | (sf << 29);
}

// A 128-wide block of K: scale copies and MMAs, in one statement.
//   copies  one scale tile of A (descriptor sa_lo) to sfa, one of B (sb_lo) to
//           sfb, PAIR: B's second (sb2_lo) to sfb + 4.  A tile fills four
//           columns, its 32 lanes repeated in all four lane quarters: column
//           c, lane l holds row 32 c + l's four scale bytes.
//   MMAs    two of K = 64 (F4) or four of K = 32, operands 32 bytes apart, into
//           d; B's scales at sfb_at.  The first adds iff `accumulate`.
// Not PAIR: by a whole converged warp, from one elected lane, the same one each
// time.  The instructions read uniform registers; a lane in a branch of its own
// moves every operand there one by one, and with few tokens that is the time
// (a stage of two copies and four MMAs 200 ns, 162 so; T = 16, N = K = 4096, 8x4
// bits: 5.3 and 4.95 us).
// PAIR: over a pair of CTAs (cta_group::2), by one lane of the even one.  A is
// 128 rows of each CTA, B half of its N rows in each, D 128 lanes x N columns in
// each; the copies run in both, from each CTA's own shared memory to its own
// tensor memory.  Here the tensor core is the time, and a whole warp that
// waits is slower (T = 8192, N = 16384, K = 4096, 4x4 bits: 190 us for 185).
template <bool F4, bool PAIR>
STRATA_DEVFN void mma_mx_block(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                               uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t sfb_at,
                               uint32_t sa_lo, uint32_t sb_lo, uint32_t sb2_lo,
                               uint32_t accumulate) {
#define STRATA_MX_CP(G, FROM, TO)       \
  "mov.b64 sd, {" FROM ", %11};\n\t"    \
  "@e tcgen05.cp.cta_group::" G ".32x128b.warpx4 [" TO "], sd;\n\t"
#define STRATA_MX_CP2(G) "add.u32 c2, %6, 4;\n\t" STRATA_MX_CP(G, "%10", "c2")
#define STRATA_MX_MMA(G, KIND, AT, ID, ACC) \
  "add.u32 a, %1, " AT ";\n\t"              \
  "add.u32 b, %2, " AT ";\n\t"              \
  "add.u32 id, %4, " ID ";\n\t"             \
  "mov.b64 ad, {a, %3};\n\t"                \
  "mov.b64 bd, {b, %3};\n\t"                \
  "@e tcgen05.mma.cta_group::" G ".kind::" KIND " [%0], ad, bd, id, [%5], [%7], " ACC ";\n\t"
#define STRATA_MX_F4(G) \
  STRATA_MX_MMA(G, "mxf4.block_scale.scale_vec::2X", "0", "0", "p") \
  STRATA_MX_MMA(G, "mxf4.block_scale.scale_vec::2X", "2", "0x40000020", "1")
#define STRATA_MX_F8(G) \
  STRATA_MX_MMA(G, "mxf8f6f4.block_scale.scale_vec::1X", "0", "0", "p") \
  STRATA_MX_MMA(G, "mxf8f6f4.block_scale.scale_vec::1X", "2", "0x20000010", "1") \
  STRATA_MX_MMA(G, "mxf8f6f4.block_scale.scale_vec::1X", "4", "0x40000020", "1") \
  STRATA_MX_MMA(G, "mxf8f6f4.block_scale.scale_vec::1X", "6", "0x60000030", "1")
#define STRATA_MX_BLOCK(G, WHO, SECOND, MMAS)                                         \
  asm volatile(                                                                       \
      "{\n\t.reg .pred e, p;\n\t.reg .b32 a, b, id, c2;\n\t.reg .b64 ad, bd, sd;\n\t" \
      "setp.ne.b32 p, %12, 0;\n\t"                                                    \
      WHO "\n\t"                                                                      \
      STRATA_MX_CP(G, "%8", "%5") STRATA_MX_CP(G, "%9", "%6") SECOND MMAS             \
      "}" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb),    \
      "r"(sfb_at), "r"(sa_lo), "r"(sb_lo), "r"(sb2_lo), "r"(kScaleDescHi),            \
      "r"(accumulate)                                                                 \
      : "memory")
  if constexpr (F4 && PAIR)
    STRATA_MX_BLOCK("2", "setp.eq.b32 e, 0, 0;", STRATA_MX_CP2("2"), STRATA_MX_F4("2"));
  else if constexpr (PAIR)
    STRATA_MX_BLOCK("2", "setp.eq.b32 e, 0, 0;", STRATA_MX_CP2("2"), STRATA_MX_F8("2"));
  else if constexpr (F4)
    STRATA_MX_BLOCK("1", "elect.sync _|e, 0xffffffff;", "", STRATA_MX_F4("1"));
  else
    STRATA_MX_BLOCK("1", "elect.sync _|e, 0xffffffff;", "", STRATA_MX_F8("1"));
#undef STRATA_MX_CP
#undef STRATA_MX_CP2
#undef STRATA_MX_MMA
#undef STRATA_MX_F4
#undef STRATA_MX_F8
#undef STRATA_MX_BLOCK
}

// A stage's copies by a whole converged warp, from one elected lane: `bytes`
// expected on `bar`, two tensor-map boxes and two runs of n bytes.
STRATA_DEVFN void load_stage_warp(uint64_t* bar, uint32_t bytes, const CUtensorMap* m0, int x0,
                                  int y0, void* d0, const CUtensorMap* m1, int x1, int y1,
                                  void* d1, const void* g2, void* d2, const void* g3, void* d3,
                                  uint32_t n) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%5], [%2, {%3, %4}], [%0];\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%9], [%6, {%7, %8}], [%0];\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%11], [%10], %14, "
      "[%0];\n\t"
      "@e cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%13], [%12], %14, "
      "[%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(bytes), "l"(reinterpret_cast<uint64_t>(m0)), "r"(x0), "r"(y0), "r"(smem_addr(d0)),
      "l"(reinterpret_cast<uint64_t>(m1)), "r"(x1), "r"(y1), "r"(smem_addr(d1)), "l"(g2),
      "r"(smem_addr(d2)), "l"(g3), "r"(smem_addr(d3)), "r"(n)
      : "memory");
}

// ---------------------------------------------------------------- CTA pairs
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
// Arrive on the barrier at `bar`'s offset in both CTAs once the tcgen05
// operations this thread has issued are complete.
STRATA_DEVFN void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// A stage's copies by a whole converged warp: four tensor-map boxes into this
// CTA's shared memory that count their bytes on a barrier of either CTA of the
// pair (`bar`: its shared::cluster address); `bytes` expected on `own` where
// that is not null.
struct PairBox {
  const CUtensorMap* map;
  int x, y;
  void* dst;
};
STRATA_DEVFN void load_stage_pair_warp(uint64_t* own, uint32_t bytes, uint32_t bar,
                                       const PairBox& a, const PairBox& b, const PairBox& c,
                                       const PairBox& d) {
#define STRATA_PAIR_LOAD(DST, MAP, X, Y)                                                       \
  "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes " \
  "[" DST "], [" MAP ", {" X ", " Y "}], [%3];\n\t"
  asm volatile(
      "{\n\t.reg .pred e, o;\n\t"
      "setp.ne.b32 o, %2, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "and.pred o, o, e;\n\t"
      "@o mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t"
      STRATA_PAIR_LOAD("%7", "%4", "%5", "%6") STRATA_PAIR_LOAD("%11", "%8", "%9", "%10")
      STRATA_PAIR_LOAD("%15", "%12", "%13", "%14") STRATA_PAIR_LOAD("%19", "%16", "%17", "%18")
      "}" ::"r"(own ? smem_addr(own) : 0u),
      "r"(bytes), "r"((uint32_t)(own != nullptr)), "r"(bar),
      "l"(reinterpret_cast<uint64_t>(a.map)), "r"(a.x), "r"(a.y), "r"(smem_addr(a.dst)),
      "l"(reinterpret_cast<uint64_t>(b.map)), "r"(b.x), "r"(b.y), "r"(smem_addr(b.dst)),
      "l"(reinterpret_cast<uint64_t>(c.map)), "r"(c.x), "r"(c.y), "r"(smem_addr(c.dst)),
      "l"(reinterpret_cast<uint64_t>(d.map)), "r"(d.x), "r"(d.y), "r"(smem_addr(d.dst))
      : "memory");
#undef STRATA_PAIR_LOAD
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
