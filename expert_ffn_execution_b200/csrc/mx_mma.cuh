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

// Instruction descriptor: both operands K-major, E8M0 scales, M = 128, N = n.
// afmt / bfmt: kind::mxf8f6f4 counts E4M3 as 0 and E2M1 as 5, kind::mxf4
// E2M1 as 1.  sf: which byte of the 32-bit scale columns the instruction's
// (first) scale is.
__host__ __device__ constexpr uint32_t idesc_mx(uint32_t afmt, uint32_t bfmt, int n, uint32_t sf) {
  return (sf << 4) | (afmt << 7) | (bfmt << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) |
         (1u << 27) | (sf << 29);
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

// ---------------------------------------------------------------- clusters
STRATA_DEVFN void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
STRATA_DEVFN uint32_t cluster_ctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
STRATA_DEVFN float ld_cluster_f32(uint32_t saddr, uint32_t rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 ra;\n\t"
      "mapa.shared::cluster.u32 ra, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [ra];\n\t}"
      : "=f"(v)
      : "r"(saddr), "r"(rank)
      : "memory");
  return v;
}

}  // namespace strata
