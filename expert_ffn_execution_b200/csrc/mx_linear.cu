// mx_linear.cu -- y[t, n] = sum_k x[t, k] w[n, k] (+ bias[n]) of two
// microscaled matrices, K contiguous in both, scales in tiles.
//
// The tensor core multiplies the codes as they are stored: tcgen05.mma with
// block scaling takes E2M1 / E4M3 codes from shared memory and the E8M0
// scales from tensor memory and sums in fp32 there, so no value is ever
// decoded.  Codes come by TMA (128-byte rows, swizzled; 4-bit weights that
// meet 8-bit activations are spread to one element a byte by the TMA itself),
// scales by plain bulk copies of whole tiles.
//
// The 128-row operand is the weights and the columns are the tokens, so a few
// tokens cost a few columns: with T tokens the call has to stream N*K codes,
// which bounds it by HBM up to a few hundred tokens.  A CTA owns 128 features
// x NT tokens; where there are fewer tiles than SMs the K axis is split over
// a cluster of up to 8 CTAs, whose partial sums are joined through
// distributed shared memory in rank order.
#include <algorithm>

#include "deal.h"
#include "mx_mma.cuh"
#include "tmap.h"

namespace strata {

namespace {

constexpr int kLThreads = 192;  // warps 0-3 epilogue, 4 copies, 5 MMA
constexpr int kLM = 128;        // features a tile
constexpr long long kLDrainCycles = 40000000LL;

template <int XF, int WF, int NT>
struct LinCfg {
  static constexpr bool F4 = XF == STRATA_MX_FP4 && WF == STRATA_MX_FP4;
  static constexpr bool kSpread = WF == STRATA_MX_FP4 && !F4;  // weights spread to bytes by TMA
  static constexpr int KS = F4 ? 256 : 128;   // K of a stage: 128 bytes of shared memory a row
  static constexpr int KI = F4 ? 64 : 32;     // K of an instruction
  static constexpr int ST = KS / 128;         // scale tiles of a stage and row block
  // what a stage's weights count on the barrier: the bytes read, spread or not
  static constexpr int WTx = kSpread ? kLM * 64 : kLM * 128;
  static constexpr int WB = kLM * 128, XB = NT * 128, SB = ST * kMxTileBytes;
  static constexpr int stage = WB + XB + 2 * SB;
  static constexpr int stride = (stage + 1023) / 1024 * 1024;
  static constexpr int S = std::min(8, (112 * 1024) / stride);  // two CTAs an SM
  static constexpr int sfcols = 8 * ST;  // tensor-memory columns of a stage's scales
  static constexpr int dcols = NT < 32 ? 32 : NT;
  static constexpr int need = dcols + S * sfcols;
  static constexpr int cols = need <= 64 ? 64 : need <= 128 ? 128 : 256;
  static_assert(need <= 256, "two CTAs share the tensor memory");
  static constexpr int smem = S * stride + 1024 + 256;
  static_assert(smem <= 115712, "two CTAs share the shared memory");
  static_assert(S >= 2 && S * stride >= NT * kLM * 4, "the partial sums fit");
};

STRATA_DEVFN void store_y(void* y, int dt, int64_t i, float v) {
  if (dt == STRATA_DTYPE_F32)
    reinterpret_cast<float*>(y)[i] = v;
  else if (dt == STRATA_DTYPE_F16)
    reinterpret_cast<__half*>(y)[i] = __float2half_rn(v);
  else
    reinterpret_cast<uint16_t*>(y)[i] = float_to_bf16_bits(v);
}

template <int XF, int WF, int NT>
__global__ void __launch_bounds__(kLThreads)
mx_linear_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                 MxLinearArgs a, int splits) {
  using C = LinCfg<XF, WF, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::S * C::stride);
  uint64_t* empty = full + C::S;
  uint64_t* tfull = empty + C::S;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* issued = reinterpret_cast<int*>(tmem_slot + 2);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = splits > 1 ? cluster_ctarank() : 0u;
  const int n0 = (int)(blockIdx.x / splits) * kLM, t0 = blockIdx.y * NT;
  const int kt = a.K / 128;                          // scale tiles of a row block
  const int chunks = (a.K + C::KS - 1) / C::KS;
  const int c0 = (int)((long long)chunks * rank / splits);
  const int nch = (int)((long long)chunks * (rank + 1) / splits) - c0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    *abort_flag = 0;
    *issued = 0;
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, C::cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  pdl_wait_prior();

  if (warp == 4) {
    if (elect_one()) {
      int i = 0;
      for (; i < nch; ++i) {
        const int s = i % C::S;
        if (!mbar_wait_guarded(&empty[s], ((i / C::S) & 1) ^ 1, a.status, abort_flag)) break;
        const int ch = c0 + i;
        const int nst = min(C::ST, kt - ch * C::ST);  // scale tiles left along K
        uint8_t* st = smem + s * C::stride;
        mbar_arrive_expect_tx(&full[s], C::WTx + C::XB + 2u * nst * kMxTileBytes);
        // coordinates in the map's elements: codes of the spread type, else bytes
        const int kw = C::kSpread ? ch * C::KS : (int)mx_row_bytes(WF, (int64_t)ch * C::KS);
        const int kx = (int)mx_row_bytes(XF, (int64_t)ch * C::KS);
        tma_load_2d(st, &wmap, kw, n0, &full[s]);
        tma_load_2d(st + C::WB, &xmap, kx, t0, &full[s]);
        bulk_g2s(st + C::WB + C::XB,
                 a.w_scales + ((int64_t)(n0 / 128) * kt + ch * C::ST) * kMxTileBytes,
                 (uint32_t)nst * kMxTileBytes, &full[s]);
        bulk_g2s(st + C::WB + C::XB + C::SB,
                 a.x_scales + ((int64_t)(t0 / 128) * kt + ch * C::ST) * kMxTileBytes,
                 (uint32_t)nst * kMxTileBytes, &full[s]);
      }
      *issued = i;
    }
    __syncwarp();
  } else if (warp == 5) {
    if (elect_one()) {
      const uint32_t hi = smem_desc_k128_hi(1024);
      const uint32_t smem0 = smem_addr(smem);
      constexpr uint32_t wf = C::F4 ? 1u : WF == STRATA_MX_FP4 ? 5u : 0u;
      constexpr uint32_t xf = C::F4 ? 1u : XF == STRATA_MX_FP4 ? 5u : 0u;
      for (int i = 0; i < nch; ++i) {
        const int s = i % C::S;
        if (!mbar_wait_guarded(&full[s], (i / C::S) & 1, a.status, abort_flag)) break;
        tc_fence_after();
        const int left = a.K - (c0 + i) * C::KS;  // a multiple of 128
        const uint32_t st = smem0 + (uint32_t)(s * C::stride);
        const uint32_t sfw = tbase + C::dcols + s * C::sfcols, sfx = sfw + 4 * C::ST;
#pragma unroll
        for (int b = 0; b < C::ST; ++b) {
          if (b * 128 < left) {
            tmem_cp_scales(sfw + 4 * b, smem_desc_scale_lo(st + C::WB + C::XB + b * kMxTileBytes));
            tmem_cp_scales(sfx + 4 * b,
                           smem_desc_scale_lo(st + C::WB + C::XB + C::SB + b * kMxTileBytes));
          }
        }
        const uint32_t wlo = smem_desc_k128_lo(st), xlo = smem_desc_k128_lo(st + C::WB);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j * C::KI < left) {
            // two instructions share a scale column at K = 64, four at K = 32
            const int b = C::F4 ? j / 2 : 0;
            const uint32_t sf = C::F4 ? 2u * (j & 1) : (uint32_t)j;
            mma_mx<C::F4>(tbase, wlo + 2 * j, xlo + 2 * j, hi, idesc_mx(wf, xf, kLM, NT, sf),
                          sfw + 4 * b, sfx + 4 * b, (uint32_t)(i + j > 0));
          }
        }
        mma_commit(&empty[s]);
      }
      mma_commit(tfull);
    }
    __syncwarp();
  } else {
    const bool ok = __all_sync(0xffffffffu, mbar_wait_guarded(tfull, 0, a.status, abort_flag) &&
                                                !*abort_flag);
    tc_fence_after();
    const int f = warp * 32 + lane;  // feature of the tile
    float* red = reinterpret_cast<float*>(smem);
    const bool mine = n0 + f < a.N;
    const float bias = ok && splits == 1 && a.bias && mine ? a.bias[n0 + f] : 0.f;
    if (ok) {
#pragma unroll 1
      for (int c = 0; c < NT; c += 16) {
        uint32_t r[16];
        tmem_ld16(tbase + ((uint32_t)(warp * 32) << 16) + c, r);
        tmem_wait_ld();
        if (splits > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) red[(c + i) * kLM + f] = __uint_as_float(r[i]);
        } else if (mine) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (t0 + c + i < a.T)
              store_y(a.y, a.y_dtype, (int64_t)(t0 + c + i) * a.ldy + n0 + f,
                      __uint_as_float(r[i]) + bias);
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // a wait gave up: every copy that was started lands, and every MMA ends,
    // before the shared and tensor memory are released (bounded)
    const int n = *issued;
    for (int s = 0; s < C::S && s < n; ++s)
      mbar_wait_bounded(&full[s], last_armed_parity(n, C::S, s), a.status, kLDrainCycles);
    mbar_wait_bounded(tfull, 0, a.status, kLDrainCycles);
  }
  __syncwarp();
  if (splits > 1) {
    cluster_sync_all();  // every rank's partial sums are written
    if (warp < 4 && n0 + (int)threadIdx.x < a.N) {
      const int f = threadIdx.x;
      const float bias = a.bias ? a.bias[n0 + f] : 0.f;
      const uint32_t base = smem_addr(smem) + 4u * f;
      for (int c = rank; c < NT && t0 + c < a.T; c += splits) {
        float v = 0.f;
        for (int q = 0; q < splits; ++q) v += ld_cluster_f32(base + 4u * kLM * c, q);
        store_y(a.y, a.y_dtype, (int64_t)(t0 + c) * a.ldy + n0 + f, v + bias);
      }
    }
    __syncwarp();
    cluster_sync_all();  // nobody leaves while its sums are read
  } else {
    __syncthreads();
  }
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tbase, C::cols);
  }
}

// Codes of a matrix as 128-byte (shared memory) x `box_rows` boxes.
bool make_mx_map(CUtensorMap* map, const uint8_t* codes, int fmt, bool spread, int rows, int K,
                 int box_rows) {
  const cuuint64_t row = (cuuint64_t)mx_row_bytes(fmt, K);
  const cuuint64_t dims[2] = {spread ? (cuuint64_t)K : row, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {row};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  return make_tmap(map, spread ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                   2, codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int XF, int WF, int NT>
cudaError_t launch_linear(const MxLinearArgs& a, cudaStream_t st) {
  using C = LinCfg<XF, WF, NT>;
  CUtensorMap wmap, xmap;
  if (!make_mx_map(&wmap, a.w_codes, WF, C::kSpread, a.N, a.K, kLM) ||
      !make_mx_map(&xmap, a.x_codes, XF, false, a.T, a.K, NT))
    return cudaErrorInvalidValue;
  const int tn = (a.N + kLM - 1) / kLM, tt = (a.T + NT - 1) / NT;
  const int chunks = (a.K + C::KS - 1) / C::KS;
  // Split K while every CTA still has two stages and the CTAs all fit at once
  int splits = 1;
  while (splits < 8 && (long long)tn * tt * splits * 2 <= 2LL * a.num_sms &&
         chunks >= splits * 2 * 2)
    splits *= 2;
  auto kern = mx_linear_kernel<XF, WF, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(tn * splits, tt);
  cfg.blockDim = dim3(kLThreads);
  cfg.dynamicSmemBytes = C::smem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, wmap, xmap, a, splits);
}

template <int XF, int WF>
cudaError_t launch_linear_t(const MxLinearArgs& a, cudaStream_t st) {
  // Token tiles of a call start at multiples of 128 (a scale tile's rows) or
  // there is one: the smallest that holds T.
  if (a.T <= 16) return launch_linear<XF, WF, 16>(a, st);
  if (a.T <= 32) return launch_linear<XF, WF, 32>(a, st);
  if (a.T <= 64) return launch_linear<XF, WF, 64>(a, st);
  if (a.T <= 128) return launch_linear<XF, WF, 128>(a, st);
  return launch_mx_gemm(a, st);
}

}  // namespace

cudaError_t launch_mx_linear(const MxLinearArgs& a, cudaStream_t st) {
  if (a.x_fmt == STRATA_MX_FP4 && a.w_fmt == STRATA_MX_FP4)
    return launch_linear_t<STRATA_MX_FP4, STRATA_MX_FP4>(a, st);
  if (a.x_fmt == STRATA_MX_FP8 && a.w_fmt == STRATA_MX_FP4)
    return launch_linear_t<STRATA_MX_FP8, STRATA_MX_FP4>(a, st);
  if (a.x_fmt == STRATA_MX_FP8 && a.w_fmt == STRATA_MX_FP8)
    return launch_linear_t<STRATA_MX_FP8, STRATA_MX_FP8>(a, st);
  return cudaErrorNotSupported;
}

}  // namespace strata
