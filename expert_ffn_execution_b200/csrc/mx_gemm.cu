// mx_gemm.cu -- the many-token form of y = x w^T over microscaled matrices.
//
// With hundreds of tokens the product is bound by how fast operands reach the
// tensor cores: an SM's share of the 4-bit rate is 61 TFLOP/s, and a tile of
// m x n spends (m + n) / 2 bytes of L2 reads per k for 2 m n operations.  So
// the tile is as large as tensor memory allows: a pair of CTAs (cta_group::2)
// multiplies 256 tokens x 256 features, each CTA loading 128 rows of both and
// holding 128 tokens x 256 features of the sums.
//
// Persistent, one pair a TPC-sized cluster: tiles in turn.  Per CTA: warps
// 0-7 read the sums out (a lane quarter of 32 tokens, half of the features
// each), warp 8 starts the copies, warp 9 of the even CTA issues the scale
// copies and the MMAs of both.  The sums of a tile (256 columns) and the
// stages' scales (12 columns per 128 of K) share the 512 columns, so the next
// tile waits until the readers have the sums in registers; they are rounded,
// turned in shared memory and stored while it runs.
#include <algorithm>

#include "deal.h"
#include "mx_mma.cuh"
#include "tmap.h"

namespace strata {

namespace {

constexpr int kGEpi = 8;                       // warps that read the sums
constexpr int kGThreads = (kGEpi + 2) * 32;
constexpr int kGM = 256, kGN = 256;            // a pair's tile
constexpr long long kGDrainCycles = 40000000LL;

template <int XF, int WF>
struct GemmCfg {
  static constexpr bool F4 = XF == STRATA_MX_FP4 && WF == STRATA_MX_FP4;
  static constexpr bool kSpread = WF == STRATA_MX_FP4 && !F4;
  static constexpr int KS = F4 ? 256 : 128, KI = F4 ? 64 : 32;
  static constexpr int ST = KS / 128;
  static constexpr int AB = 128 * 128, BB = 128 * 128;           // a CTA's rows of x and w
  static constexpr int BTx = kSpread ? BB / 2 : BB;              // bytes read, spread or not
  static constexpr int SA = ST * kMxTileBytes, SBb = 2 * SA;     // scales of 128 and 256 rows
  static constexpr int stage = AB + BB + SA + SBb;
  static constexpr int stride = (stage + 1023) / 1024 * 1024;
  static constexpr int epi = kGEpi * 32 * 64;
  static constexpr int S = (227 * 1024 - 2048 - epi) / stride;
  static constexpr int smem = S * stride + epi + 2048;
  static constexpr int sfcols = 12 * ST;
  static_assert(kGN + S * sfcols <= 512, "sums and scales fit the tensor memory");
};

template <int XF, int WF, int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGThreads, 1)
mx_gemm_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap wmap,
               const __grid_constant__ CUtensorMap xsmap, const __grid_constant__ CUtensorMap wsmap,
               MxLinearArgs a, int mt, int tiles, int vec) {
  using C = GemmCfg<XF, WF>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* epi = smem + C::S * C::stride;
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + C::epi);
  uint64_t* empty = full + C::S;
  uint64_t* tfull = empty + C::S;
  uint64_t* tempty = tfull + 1;
  uint64_t* done = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* issued = reinterpret_cast<int*>(tmem_slot + 2);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const int chunks = (a.K + C::KS - 1) / C::KS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 2 * kGEpi);
    mbar_init(done, 1);
    *abort_flag = 0;
    *issued = 0;
    fence_barrier_init();
  }
  if (warp == kGEpi + 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_relaxed();  // both CTAs' barriers and tensor memory are ready
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  pdl_wait_prior();

  if (warp == kGEpi) {
    // ------------------------------------------------ copies, counted on the even CTA's barriers
    if (elect_one()) {
      int i = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += pairs) {
        const int t0 = (tile % mt) * kGM, n0 = (tile / mt) * kGN;
        for (int ch = 0; ch < chunks; ++ch, ++i) {
          const int s = i % C::S;
          if (!mbar_wait_guarded(&empty[s], ((i / C::S) & 1) ^ 1, a.status, abort_flag)) {
            ok = false;
            break;
          }
          if (rank == 0)
            mbar_arrive_expect_tx(&full[s], 2u * (C::AB + C::BTx + C::SA + C::SBb));
          uint8_t* st = smem + s * C::stride;
          const uint32_t bar = cluster_addr(smem_addr(&full[s]), 0);
          const int kx = (int)mx_row_bytes(XF, (int64_t)ch * C::KS);
          const int kw = C::kSpread ? ch * C::KS : (int)mx_row_bytes(WF, (int64_t)ch * C::KS);
          tma_load_2d_pair(st, &xmap, kx, t0 + 128 * (int)rank, bar);
          tma_load_2d_pair(st + C::AB, &wmap, kw, n0 + 128 * (int)rank, bar);
          tma_load_2d_pair(st + C::AB + C::BB, &xsmap, ch * C::ST * 64, t0 / 128 + (int)rank, bar);
          tma_load_2d_pair(st + C::AB + C::BB + C::SA, &wsmap, ch * C::ST * 64, n0 / 128, bar);
        }
      }
      *issued = i;
    }
    __syncwarp();
  } else if (warp == kGEpi + 1) {
    // ------------------------------------------------ MMAs, by the even CTA for both
    if (rank == 0 && elect_one()) {
      const uint32_t hi = smem_desc_k128_hi(1024);
      const uint32_t smem0 = smem_addr(smem);
      constexpr uint32_t xf = C::F4 ? 1u : XF == STRATA_MX_FP4 ? 5u : 0u;
      constexpr uint32_t wf = C::F4 ? 1u : WF == STRATA_MX_FP4 ? 5u : 0u;
      int i = 0, it = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += pairs, ++it) {
        ok = mbar_wait_guarded(tempty, (it & 1) ^ 1, a.status, abort_flag);
        tc_fence_after();
        for (int ch = 0; ch < chunks && ok; ++ch, ++i) {
          const int s = i % C::S;
          ok = mbar_wait_guarded(&full[s], (i / C::S) & 1, a.status, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const int left = a.K - ch * C::KS;  // a multiple of 128
          const uint32_t st = smem0 + (uint32_t)(s * C::stride);
          const uint32_t ssa = st + C::AB + C::BB, ssb = ssa + C::SA;
          const uint32_t sfx = tbase + kGN + s * C::sfcols, sfw = sfx + 4 * C::ST;
#pragma unroll
          for (int b = 0; b < C::ST; ++b) {
            tmem_cp_scales_pair(sfx + 4 * b, smem_desc_scale_lo(ssa + b * kMxTileBytes));
#pragma unroll
            for (int r = 0; r < 2; ++r)
              tmem_cp_scales_pair(sfw + 8 * b + 4 * r,
                                  smem_desc_scale_lo(ssb + (r * C::ST + b) * kMxTileBytes));
          }
          const uint32_t xlo = smem_desc_k128_lo(st), wlo = smem_desc_k128_lo(st + C::AB);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j * C::KI < left) {
              const int b = C::F4 ? j / 2 : 0;
              const uint32_t sf = C::F4 ? 2u * (j & 1) : (uint32_t)j;
              mma_mx_pair<C::F4>(tbase, xlo + 2 * j, wlo + 2 * j, hi, idesc_mx(xf, wf, kGM, kGN, sf),
                                 sfx + 4 * b, sfw + 8 * b, (uint32_t)(ch + j > 0));
            }
          }
          mma_commit_pair(&empty[s]);
        }
        if (ok) mma_commit_pair(tfull);
      }
      mma_commit_pair(done);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ sums -> y
    const int q = warp % 4, half = warp / 4;
    uint8_t* buf = epi + warp * (32 * 64);
    const uint32_t lead = cluster_addr(smem_addr(tempty), 0);
    constexpr int kEl = DT == STRATA_DTYPE_F32 ? 4 : 2;
    constexpr int kPer = 64 / kEl;   // features a pass
    int it = 0;
    for (int tile = pair; tile < tiles; tile += pairs, ++it) {
      const int t0 = (tile % mt) * kGM + 128 * (int)rank + 32 * q;
      const int n0 = (tile / mt) * kGN + 128 * half;
      const bool ok = mbar_wait_guarded(tfull, it & 1, a.status, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      uint32_t r[128];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_ld32(tbase + ((uint32_t)(q * 32) << 16) + 128 * half + 32 * c, r + 32 * c);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(lead);
      if (a.bias) {
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (n0 + i < a.N) r[i] = __float_as_uint(__uint_as_float(r[i]) + a.bias[n0 + i]);
      }
      if constexpr (kEl == 2) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
          r[i] = pack2<DT>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
      }
      // 64 bytes of each of the 32 rows at a time through shared memory, the
      // 16-byte pieces of row r at places piece ^ (r/2 % 4): both the writes
      // (a row a lane) and the reads (four lanes a row) touch every bank once
      const int rows = min(32, a.T - t0);
      uint8_t* const yb = reinterpret_cast<uint8_t*>(a.y) + ((int64_t)t0 * a.ldy + n0) * kEl;
      const bool whole = vec && n0 + 128 <= a.N && rows > 0;
      const int row = lane / 4, pc = lane % 4;
#pragma unroll
      for (int p = 0; p < 128 / kPer; ++p) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(buf + lane * 64 + ((i ^ (lane / 2)) & 3) * 16) =
              make_uint4(r[16 * p + 4 * i], r[16 * p + 4 * i + 1], r[16 * p + 4 * i + 2],
                         r[16 * p + 4 * i + 3]);
        __syncwarp();
        if (whole) {
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (g * 8 + row < rows)
              *reinterpret_cast<uint4*>(yb + (int64_t)(g * 8 + row) * a.ldy * kEl + p * 64 +
                                        pc * 16) =
                  *reinterpret_cast<const uint4*>(buf + (g * 8 + row) * 64 +
                                                  ((pc ^ (row / 2)) & 3) * 16);
        } else {
          // rows without 16-byte boundaries, or the last features: a lane a feature
          const int left = min(kPer, a.N - n0 - p * kPer);
#pragma unroll 1
          for (int w = 0; w < rows; ++w) {
            if (lane >= left) continue;
            const int at = lane * kEl;
            const uint8_t* src = buf + w * 64 + (((at / 16) ^ (w / 2)) & 3) * 16 + at % 16;
            uint8_t* dst = yb + (int64_t)w * a.ldy * kEl + p * 64 + at;
            if constexpr (kEl == 4)
              *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
            else
              *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(src);
          }
        }
      }
    }
  }
  // the even CTA's MMAs read both CTAs' shared memory: all are done, and after
  // a wait that gave up all copies have landed, before either CTA goes on
  __syncthreads();
  if (threadIdx.x == 0) {
    mbar_wait_bounded(done, 0, a.status);
    if (*abort_flag && rank == 0) {
      const int n = *issued;
      for (int s = 0; s < C::S && s < n; ++s)
        mbar_wait_bounded(&full[s], last_armed_parity(n, C::S, s), a.status, kGDrainCycles);
    }
  }
  __syncthreads();
  cluster_sync_relaxed();
  if (warp == kGEpi + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, 512);
  }
}

bool make_code_map(CUtensorMap* map, const uint8_t* codes, int fmt, bool spread, int rows, int K) {
  const cuuint64_t row = (cuuint64_t)mx_row_bytes(fmt, K);
  const cuuint64_t dims[2] = {spread ? (cuuint64_t)K : row, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {row};
  const cuuint32_t box[2] = {128, 128};
  return make_tmap(map, spread ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8,
                   2, codes, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scale tiles as 64-bit words: a row of tiles a row, boxes of `st` tiles x
// `box_rows` rows; tiles behind the last read as 0.
bool make_scale_map(CUtensorMap* map, const uint8_t* scales, int rows, int K, int st,
                    int box_rows) {
  const cuuint64_t row = (cuuint64_t)(K / 128) * kMxTileBytes;
  const cuuint64_t dims[2] = {row / 8, (cuuint64_t)mx_ceil(rows, kMxTileRows)};
  const cuuint64_t strides[1] = {row};
  const cuuint32_t box[2] = {(cuuint32_t)(st * kMxTileBytes / 8), (cuuint32_t)box_rows};
  return make_tmap(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, 2, scales, dims, strides, box,
                   CU_TENSOR_MAP_SWIZZLE_NONE);
}

template <int XF, int WF, int DT>
cudaError_t launch_gemm(const MxLinearArgs& a, cudaStream_t st) {
  using C = GemmCfg<XF, WF>;
  CUtensorMap xmap, wmap, xsmap, wsmap;
  if (!make_code_map(&xmap, a.x_codes, XF, false, a.T, a.K) ||
      !make_code_map(&wmap, a.w_codes, WF, C::kSpread, a.N, a.K) ||
      !make_scale_map(&xsmap, a.x_scales, a.T, a.K, C::ST, 1) ||
      !make_scale_map(&wsmap, a.w_scales, a.N, a.K, C::ST, 2))
    return cudaErrorInvalidValue;
  const int mt = (a.T + kGM - 1) / kGM, nt = (a.N + kGN - 1) / kGN;
  const int tiles = mt * nt;
  constexpr int el = DT == STRATA_DTYPE_F32 ? 4 : 2;
  const int vec = (reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && a.ldy * el % 16 == 0) ? 1 : 0;
  auto kern = mx_gemm_kernel<XF, WF, DT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(2 * std::min(tiles, a.num_sms / 2));
  cfg.blockDim = dim3(kGThreads);
  cfg.dynamicSmemBytes = C::smem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, xmap, wmap, xsmap, wsmap, a, mt, tiles, vec);
}

template <int XF, int WF>
cudaError_t launch_gemm_y(const MxLinearArgs& a, cudaStream_t st) {
  if (a.y_dtype == STRATA_DTYPE_F32) return launch_gemm<XF, WF, STRATA_DTYPE_F32>(a, st);
  if (a.y_dtype == STRATA_DTYPE_F16) return launch_gemm<XF, WF, STRATA_DTYPE_F16>(a, st);
  return launch_gemm<XF, WF, STRATA_DTYPE_BF16>(a, st);
}

}  // namespace

cudaError_t launch_mx_gemm(const MxLinearArgs& a, cudaStream_t st) {
  if (a.x_fmt == STRATA_MX_FP4) return launch_gemm_y<STRATA_MX_FP4, STRATA_MX_FP4>(a, st);
  if (a.w_fmt == STRATA_MX_FP4) return launch_gemm_y<STRATA_MX_FP8, STRATA_MX_FP4>(a, st);
  return launch_gemm_y<STRATA_MX_FP8, STRATA_MX_FP8>(a, st);
}

}  // namespace strata
