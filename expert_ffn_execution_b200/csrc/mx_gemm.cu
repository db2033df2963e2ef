// mx_gemm.cu -- the many-token form of y = x w^T over microscaled matrices.
//
// With hundreds of tokens the product is bound by how fast operands reach the
// tensor cores: a tile of m x n reads (m + n) K elements from L2 for 2 m n K
// operations, and the 148 SMs together get 11 to 13 TB/s.  So the tile is as
// large as tensor memory allows: a pair of CTAs (cta_group::2) multiplies 256
// rows of A x 256 of B, each CTA loading 128 of both and holding 128 x 256 of
// the sums.  T = 8192, N = 16384, K = 4096, 4x4 bits: 431 us with 128 x 128 tiles
// of one CTA, 187 us (5.9 PFLOP/s) here; N = 10240, K = 2560, 8x4 bits: 304 and
// 142 us (3.0 PFLOP/s); the tensor pipe is active for 74 and 79 % of the cycles.
// In a loop of seconds power is the bound (216 and 166 us).  The order of the
// tiles makes no difference (operands of this size stay in L2).
//
// Persistent: a pair takes tiles in turn.  Per CTA: warps 0-7 read the sums
// out (a lane quarter of 32 rows of A, half of B's each), warp 8 starts the
// copies, a lane of warp 9 of the even CTA issues the scale copies and the MMAs
// of both.  The sums of a tile (256 columns) and the stages' scales (12 columns
// per 128 of K) share the 512 columns, so the next tile waits until the
// readers have the sums in registers (500 cycles after the last MMA); they are
// rounded and stored while it runs.  Halves of 128 columns in three rotating
// buffers, which need not wait, are slower (229 us when one buffer took 206):
// an MMA of 128 columns reads its other operand twice as often.
#include <algorithm>

#include "deal.h"
#include "mx_mma.cuh"
#include "mx_plan.h"
#include "tmap.h"

namespace strata {

namespace {

constexpr int kGEpi = 8;                       // warps that read the sums
constexpr int kGThreads = (kGEpi + 2) * 32;
constexpr int kGM = 256, kGN = 256;            // a pair's tile
constexpr long long kGDrainCycles = 40000000LL;

// Which matrix is A decides what a lane of the tensor memory is when the sums
// are read.  A feature (A = w): a token's 32 features are one store of the warp,
// on any alignment, in few instructions.  A token (WIDE, A = x): rows are turned
// in shared memory and stored 16 bytes a lane.  The first ends a tile sooner
// (T = 1452, N = 25296, K = 640, 4x4 bits: 22 us for 29; T = 2048, N = K = 4096:
// 16.0 for 17.3), the second takes less of the power that bounds long calls
// (T = 8192, N = 10240, K = 2560, 8x4 bits, in a loop: 164 us for 173).
template <int XF, int WF, bool WIDE>
struct GemmCfg {
  static constexpr bool F4 = XF == STRATA_MX_FP4 && WF == STRATA_MX_FP4;
  static constexpr int AF = WIDE ? XF : WF, BF = WIDE ? WF : XF;
  static constexpr bool spread(int fmt) { return fmt == STRATA_MX_FP4 && !F4; }
  static constexpr int KS = F4 ? 256 : 128;
  static constexpr int ST = KS / 128;
  static constexpr int AB = 128 * 128;                           // a CTA's rows of A, and of B
  static constexpr int tx(int fmt) { return spread(fmt) ? AB / 2 : AB; }  // bytes read
  static constexpr int SA = ST * kMxTileBytes, SBb = 2 * SA;     // scales of 128 and 256 rows
  static constexpr int stage = 2 * AB + SA + SBb;
  static constexpr int stride = (stage + 1023) / 1024 * 1024;
  static constexpr int epi = WIDE ? kGEpi * 32 * 64 : 0;         // 64 bytes of 32 rows a warp
  static constexpr int bias = WIDE ? kGEpi * 128 * 4 : 0;
  static constexpr int S = (227 * 1024 - 2048 - epi - bias) / stride;
  static constexpr int smem = S * stride + epi + bias + 2048;
  static constexpr int sfcols = 12 * ST;
  // how the MMA's descriptor counts a format, and the map's x of a chunk
  static constexpr uint32_t kind(int fmt) { return F4 ? 1u : fmt == STRATA_MX_FP4 ? 5u : 0u; }
  STRATA_DEVFN static int at(int fmt, int ch) {
    return spread(fmt) ? ch * KS : (int)mx_row_bytes(fmt, (int64_t)ch * KS);
  }
  static_assert(kGN + S * sfcols <= 512, "sums and scales fit the tensor memory");
};

// 128 tokens of the lane's feature -> y, `count` of them y's, rows `pitch`
// bytes apart.  A token's store is 32 features side by side, on any alignment.
template <int DT, bool WHOLE>
STRATA_DEVFN void store_tokens(uint8_t* y, int64_t pitch, const uint32_t (&r)[128], float bias,
                               int count) {
#pragma unroll
  for (int k = 0; k < 128; ++k, y += pitch) {
    const float v = __uint_as_float(r[k]) + bias;
    if (WHOLE || k < count) {
      if constexpr (DT == STRATA_DTYPE_F32)
        *reinterpret_cast<float*>(y) = v;
      else
        *reinterpret_cast<uint16_t*>(y) = (uint16_t)pack2<DT>(v, v);
    }
  }
}

// A pass's 64 bytes of `rows` rows, a word a lane, side by side, where rows end
// inside (`left` bytes of them are y's).
template <int EL>
STRATA_DEVFN void store_rows(const uint8_t* buf, uint8_t* y, int64_t pitch, int rows, int left,
                             int lane) {
  const int at = lane % 16 * 4;
  if (at >= left) return;
#pragma unroll 4
  for (int g = 0; g < 16; ++g) {
    const int row = g * 2 + lane / 16;
    const uint8_t* src = buf + row * 64 + (((at / 16) ^ (row / 2)) & 3) * 16 + at % 16;
    uint8_t* dst = y + row * pitch + at;
    if (row < rows) {
      if (EL == 4 || at + 4 <= left)
        *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(src);
      else  // the first of the last pair
        *reinterpret_cast<uint16_t*>(dst) = *reinterpret_cast<const uint16_t*>(src);
    }
  }
}

template <int XF, int WF, int DT, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGThreads, 1)
mx_gemm_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
               const __grid_constant__ CUtensorMap asmap, const __grid_constant__ CUtensorMap bsmap,
               MxLinearArgs a, int mt, int tiles) {
  using C = GemmCfg<XF, WF, WIDE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* epi = smem + C::S * C::stride;
  float* bias_s = reinterpret_cast<float*>(epi + C::epi);
  uint64_t* full = reinterpret_cast<uint64_t*>(epi + C::epi + C::bias);
  uint64_t* empty = full + C::S;
  uint64_t* tfull = empty + C::S;
  uint64_t* tempty = tfull + 1;
  uint64_t* done = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* issued = reinterpret_cast<int*>(tmem_slot + 2);

  // the warp from one lane: known to be the same in all, as is what follows from it
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
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
  const uint32_t tbase = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  pdl_wait_prior();

  if (warp == kGEpi) {
    // ------------------------------------------------ copies, counted on the even CTA's barriers
    int i = 0, s = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int tile = pair; tile < tiles && ok; tile += pairs) {
      const int tt = (tile % mt) * 256, tn = (tile / mt) * 256;  // its tokens and features
      const int a0 = WIDE ? tt : tn, b0 = WIDE ? tn : tt;
      for (int ch = 0; ch < chunks; ++ch, ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait_guarded(&empty[s], ph, a.status, abort_flag));
        if (!ok) break;
        uint8_t* st = smem + s * C::stride;
        load_stage_pair_warp(
            rank == 0 ? &full[s] : nullptr, 2u * (C::tx(C::AF) + C::tx(C::BF) + C::SA + C::SBb),
            cluster_addr(smem_addr(&full[s]), 0),
            {&amap, C::at(C::AF, ch), a0 + 128 * (int)rank, st},
            {&bmap, C::at(C::BF, ch), b0 + 128 * (int)rank, st + C::AB},
            {&asmap, ch * C::ST * 64, a0 / 128 + (int)rank, st + 2 * C::AB},
            {&bsmap, ch * C::ST * 64, b0 / 128, st + 2 * C::AB + C::SA});
        if (++s == C::S) s = 0, ph ^= 1u;
      }
    }
    *issued = i;
    __syncwarp();
  } else if (warp == kGEpi + 1) {
    // ------------------------------------------------ MMAs, by the even CTA for both
    if (rank == 0 && elect_one()) {
      const uint32_t hi = smem_desc_k128_hi(1024);
      const uint32_t smem0 = smem_addr(smem);
      int s = 0, it = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int tile = pair; tile < tiles && ok; tile += pairs, ++it) {
        ok = mbar_wait_guarded(tempty, (it & 1) ^ 1, a.status, abort_flag);
        tc_fence_after();
        for (int ch = 0; ch < chunks && ok; ++ch) {
          ok = mbar_wait_guarded(&full[s], ph, a.status, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const int left = a.K - ch * C::KS;  // a multiple of 128
          const uint32_t st = smem0 + (uint32_t)(s * C::stride);
          const uint32_t ssa = st + 2 * C::AB, ssb = ssa + C::SA;
          const uint32_t sfa = tbase + kGN + s * C::sfcols, sfb = sfa + 4 * C::ST;
          const uint32_t alo = smem_desc_k128_lo(st), blo = smem_desc_k128_lo(st + C::AB);
#pragma unroll
          for (int b = 0; b < C::ST; ++b) {
            if (b * 128 < left) {
              const uint32_t sb = ssb + b * kMxTileBytes;  // of the first 128 rows of B
              mma_mx_block<C::F4, true>(
                  tbase, alo + 4 * b, blo + 4 * b, hi,
                  idesc_mx(C::kind(C::AF), C::kind(C::BF), kGM, kGN, 0), sfa + 4 * b, sfb + 8 * b,
                  sfb + 8 * b, smem_desc_scale_lo(ssa + b * kMxTileBytes), smem_desc_scale_lo(sb),
                  smem_desc_scale_lo(sb + C::SA), (uint32_t)(ch + b > 0));
            }
          }
          mma_commit_pair(&empty[s]);
          if (++s == C::S) s = 0, ph ^= 1u;
        }
        if (ok) mma_commit_pair(tfull);
      }
      mma_commit_pair(done);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ sums -> y
    const int q = warp % 4, half = warp / 4;  // 32 rows of A, 128 of B
    const uint32_t lead = cluster_addr(smem_addr(tempty), 0);
    constexpr int kEl = DT == STRATA_DTYPE_F32 ? 4 : 2;
    constexpr int kPer = 64 / kEl;  // features a pass of WIDE
    uint8_t* const buf = epi + warp * 32 * 64;
    int it = 0;
    for (int tile = pair; tile < tiles; tile += pairs, ++it) {
      const int in_a = 128 * (int)rank + 32 * q, in_b = 128 * half;
      const int t0 = (tile % mt) * 256 + (WIDE ? in_a : in_b);
      const int n0 = (tile / mt) * 256 + (WIDE ? in_b : in_a);
      float bias = 0.f;
      float* const bs = bias_s + warp * 128;
      if (WIDE && a.bias) {  // this warp's 128 features' while the MMAs run
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = n0 + 32 * i + lane;
          bs[32 * i + lane] = n < a.N ? a.bias[n] : 0.f;
        }
      } else if (a.bias && n0 + lane < a.N) {
        bias = a.bias[n0 + lane];
      }
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
      if constexpr (!WIDE) {
        if (n0 + lane < a.N) {
          uint8_t* const y = reinterpret_cast<uint8_t*>(a.y) + ((int64_t)t0 * a.ldy + n0 + lane) * kEl;
          if (t0 + 128 <= a.T)
            store_tokens<DT, true>(y, a.ldy * kEl, r, bias, 128);
          else
            store_tokens<DT, false>(y, a.ldy * kEl, r, bias, a.T - t0);
        }
        __syncwarp();
      } else {
        if (a.bias) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float4 b = reinterpret_cast<const float4*>(bs)[i];
            r[4 * i] = __float_as_uint(__uint_as_float(r[4 * i]) + b.x);
            r[4 * i + 1] = __float_as_uint(__uint_as_float(r[4 * i + 1]) + b.y);
            r[4 * i + 2] = __float_as_uint(__uint_as_float(r[4 * i + 2]) + b.z);
            r[4 * i + 3] = __float_as_uint(__uint_as_float(r[4 * i + 3]) + b.w);
          }
        }
        if constexpr (kEl == 2) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            r[i] = pack2<DT>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        }
        const int rows = min(32, a.T - t0);
        uint8_t* const yb = reinterpret_cast<uint8_t*>(a.y) + ((int64_t)t0 * a.ldy + n0) * kEl;
        // 64 bytes of each of the 32 rows at a time through shared memory, the
        // 16-byte pieces of row r at places piece ^ (r/2 % 4): both the writes
        // (a row a lane) and the reads (four lanes a row) touch every bank once
        const bool whole = n0 + 128 <= a.N;
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
            store_rows<kEl>(buf, yb + p * 64, a.ldy * kEl, rows, (a.N - n0 - p * kPer) * kEl, lane);
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

template <int XF, int WF, int DT, bool WIDE>
cudaError_t launch_gemm(const MxLinearArgs& a, cudaStream_t st) {
  using C = GemmCfg<XF, WF, WIDE>;
  CUtensorMap xmap, wmap, xsmap, wsmap;
  if (!make_code_map(&xmap, a.x_codes, XF, C::spread(XF), a.T, a.K) ||
      !make_code_map(&wmap, a.w_codes, WF, C::spread(WF), a.N, a.K) ||
      !make_scale_map(&xsmap, a.x_scales, a.T, a.K, C::ST, WIDE ? 1 : 2) ||
      !make_scale_map(&wsmap, a.w_scales, a.N, a.K, C::ST, WIDE ? 2 : 1))
    return cudaErrorInvalidValue;
  const int mt = (a.T + 255) / 256, nt = (a.N + 255) / 256;
  const int tiles = mt * nt;
  auto kern = mx_gemm_kernel<XF, WF, DT, WIDE>;
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
  return WIDE ? cudaLaunchKernelEx(&cfg, kern, xmap, wmap, xsmap, wsmap, a, mt, tiles)
              : cudaLaunchKernelEx(&cfg, kern, wmap, xmap, wsmap, xsmap, a, mt, tiles);
}

template <int XF, int WF, int DT>
cudaError_t launch_gemm_rows(const MxLinearArgs& a, cudaStream_t st) {
  constexpr int el = DT == STRATA_DTYPE_F32 ? 4 : 2;
  const bool aligned = reinterpret_cast<uintptr_t>(a.y) % 16 == 0 && a.ldy * el % 16 == 0;
  return plan_wide(a.T, a.N, a.K, GemmCfg<XF, WF, true>::F4, aligned, a.num_sms)
             ? launch_gemm<XF, WF, DT, true>(a, st)
             : launch_gemm<XF, WF, DT, false>(a, st);
}

template <int XF, int WF>
cudaError_t launch_gemm_y(const MxLinearArgs& a, cudaStream_t st) {
  if (a.y_dtype == STRATA_DTYPE_F32) return launch_gemm_rows<XF, WF, STRATA_DTYPE_F32>(a, st);
  if (a.y_dtype == STRATA_DTYPE_F16) return launch_gemm_rows<XF, WF, STRATA_DTYPE_F16>(a, st);
  return launch_gemm_rows<XF, WF, STRATA_DTYPE_BF16>(a, st);
}

}  // namespace

cudaError_t launch_mx_gemm(const MxLinearArgs& a, cudaStream_t st) {
  if (a.x_fmt == STRATA_MX_FP4) return launch_gemm_y<STRATA_MX_FP4, STRATA_MX_FP4>(a, st);
  if (a.w_fmt == STRATA_MX_FP4) return launch_gemm_y<STRATA_MX_FP8, STRATA_MX_FP4>(a, st);
  return launch_gemm_y<STRATA_MX_FP8, STRATA_MX_FP8>(a, st);
}

}  // namespace strata
