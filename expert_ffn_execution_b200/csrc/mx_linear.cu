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
constexpr int kLBatch = 2;      // joined pieces in flight a thread
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
  static constexpr int sfcols = 8 * ST;  // tensor-memory columns of a stage's scales
  static constexpr int dcols = NT < 32 ? 32 : NT;
  static constexpr int head = 1024;      // barriers, and the alignment of what follows
  // Stages of a CTA that has its SM to itself, and of one that shares it with
  // another (shared memory, and with it tensor memory, split in two).
  static constexpr int S1 = (227 * 1024 - head - 1024) / stride;
  static constexpr int S2 = (113 * 1024 - head - 1024) / stride;
  static constexpr int smem(int S) { return S * stride + head + 1024; }
  static constexpr int cols(int S) {
    return dcols + S * sfcols <= 64 ? 64 : dcols + S * sfcols <= 128 ? 128 : 256;
  }
  static_assert(dcols + S1 * sfcols <= 256, "at most half of the tensor memory");
  static_assert(S2 >= 2 && S2 * stride >= NT * kLM * 4, "the partial sums fit");
  static_assert((2 * S1 + 1) * 8 + 16 <= head, "the barriers fit");
};

// Four consecutive values of a row of y; `vec`: the row's pieces of four are
// aligned for one store.
template <int DT>
STRATA_DEVFN void store4(void* y, int64_t i, const float (&v)[4], int n, bool vec) {
  if constexpr (DT == STRATA_DTYPE_F32) {
    float* p = reinterpret_cast<float*>(y) + i;
    if (vec && n == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < n) p[k] = v[k];
    }
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(y) + i;
    const uint32_t lo = pack2<DT>(v[0], v[1]), hi = pack2<DT>(v[2], v[3]);
    if (vec && n == 4) {
      *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < n) p[k] = (uint16_t)((k < 2 ? lo : hi) >> (16 * (k & 1)));
    }
  }
}

// The ranks' sums -> y.  Rank r joins tokens r, r + splits, ...: a thread four
// features of one, kLBatch of them at a time with all ranks' loads in flight.
template <int DT, int NT>
STRATA_DEVFN void write_y(const MxLinearArgs& a, const uint8_t* smem, int n0, int t0, int rank,
                          int splits) {
  constexpr int kEl = DT == STRATA_DTYPE_F32 ? 4 : 2;
  const int nt = min(NT, a.T - t0);
  const int items = nt > rank ? ((nt - rank - 1) / splits + 1) * (kLM / 4) : 0;
  const uint32_t base = smem_addr(smem);
  const bool vec = a.ldy % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % (4 * kEl) == 0;
  // a thread's feature is the same in all of its items
  static_assert(kLThreads % 32 == 0, "items of a thread are whole tokens apart");
  const int f = threadIdx.x % 32 * 4, n = n0 + f, left = min(4, a.N - n);
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.bias) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < left) bias[k] = a.bias[n + k];
  }
  void* const y = a.y;
  if (splits == 1) {
#pragma unroll 1
    for (int i = threadIdx.x; i < items; i += kLThreads) {
      const float4 v = *reinterpret_cast<const float4*>(smem + 4u * (uint32_t)((i / 32) * kLM + f));
      const float s[4] = {v.x + bias[0], v.y + bias[1], v.z + bias[2], v.w + bias[3]};
      store4<DT>(y, (int64_t)(t0 + i / 32) * a.ldy + n, s, left, vec);
    }
    return;
  }
#pragma unroll 1
  for (int i0 = threadIdx.x; i0 < items; i0 += kLThreads * kLBatch) {
    float4 v[kLBatch][8];
#pragma unroll
    for (int b = 0; b < kLBatch; ++b) {
      const int i = i0 + b * kLThreads;
      const uint32_t at = base + 4u * (uint32_t)((rank + (i / 32) * splits) * kLM + f);
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < splits && i < items) v[b][q] = ld_cluster_f32x4(cluster_addr(at, q));
    }
#pragma unroll
    for (int b = 0; b < kLBatch; ++b) {
      const int i = i0 + b * kLThreads;
      if (i >= items) break;
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (q < splits) {
          s[0] += v[b][q].x;
          s[1] += v[b][q].y;
          s[2] += v[b][q].z;
          s[3] += v[b][q].w;
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += bias[k];
      store4<DT>(y, (int64_t)(t0 + rank + (i / 32) * splits) * a.ldy + n, s, left, vec);
    }
  }
}

template <int XF, int WF, int NT>
__global__ void __launch_bounds__(kLThreads)
mx_linear_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                 MxLinearArgs a, int splits, int S) {
  using C = LinCfg<XF, WF, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem0 =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* smem = smem0 + C::head;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem0);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
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
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    *abort_flag = 0;
    *issued = 0;
    fence_barrier_init();
  }
  if (warp == 4 && lane == 0) {
    prefetch_tensormap(&wmap);
    prefetch_tensormap(&xmap);
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, C::cols(S));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  pdl_wait_prior();

  if (warp == 4) {
    if (elect_one()) {
      int i = 0, s = 0;
      uint32_t ph = 1;
      for (; i < nch; ++i) {
        if (!mbar_wait_guarded(&empty[s], ph, a.status, abort_flag)) break;
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
        if (++s == S) s = 0, ph ^= 1u;
      }
      *issued = i;
    }
    __syncwarp();
  } else if (warp == 5) {
    if (elect_one()) {
      const uint32_t hi = smem_desc_k128_hi(1024);
      const uint32_t stages = smem_addr(smem);
      constexpr uint32_t wf = C::F4 ? 1u : WF == STRATA_MX_FP4 ? 5u : 0u;
      constexpr uint32_t xf = C::F4 ? 1u : XF == STRATA_MX_FP4 ? 5u : 0u;
      int s = 0;
      uint32_t ph = 0;
      for (int i = 0; i < nch; ++i) {
        if (!mbar_wait_guarded(&full[s], ph, a.status, abort_flag)) break;
        tc_fence_after();
        const int left = a.K - (c0 + i) * C::KS;  // a multiple of 128
        const uint32_t st = stages + (uint32_t)(s * C::stride);
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
        if (++s == S) s = 0, ph ^= 1u;
      }
      mma_commit(tfull);
    }
    __syncwarp();
  } else {
    const bool ok = __all_sync(0xffffffffu, mbar_wait_guarded(tfull, 0, a.status, abort_flag) &&
                                                !*abort_flag);
    tc_fence_after();
    // sums -> shared memory [token][feature], over the stages
    float* red = reinterpret_cast<float*>(smem);
    const int f = warp * 32 + lane;
    if (ok) {
#pragma unroll 1
      for (int c = 0; c < NT && t0 + c < a.T; c += 16) {
        uint32_t r[16];
        tmem_ld16(tbase + ((uint32_t)(warp * 32) << 16) + c, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) red[(c + i) * kLM + f] = __uint_as_float(r[i]);
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // a wait gave up: every copy that was started lands, and every MMA ends,
    // before the shared and tensor memory are released (bounded)
    const int n = *issued;
    for (int s = 0; s < S && s < n; ++s)
      mbar_wait_bounded(&full[s], last_armed_parity(n, S, s), a.status, kLDrainCycles);
    mbar_wait_bounded(tfull, 0, a.status, kLDrainCycles);
  }
  __syncwarp();
  if (splits > 1) cluster_sync_all();  // every rank's sums are written
  if (a.y_dtype == STRATA_DTYPE_F32)
    write_y<STRATA_DTYPE_F32, NT>(a, smem, n0, t0, rank, splits);
  else if (a.y_dtype == STRATA_DTYPE_F16)
    write_y<STRATA_DTYPE_F16, NT>(a, smem, n0, t0, rank, splits);
  else
    write_y<STRATA_DTYPE_BF16, NT>(a, smem, n0, t0, rank, splits);
  __syncwarp();
  if (splits > 1) cluster_sync_relaxed();  // nobody leaves while its sums are read
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tbase, C::cols(S));
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
  // Split K where that ends sooner.  A stage costs its SM its 128-byte rows
  // (about 0.2 us at 16 tokens: 2.5 cycles a row), whichever CTA it belongs
  // to; joining costs about 9 such stages and one more for 8 tokens.  N =
  // 2560, K = 8192, T = 4, 8x4 bits: 16.0, 11.0, 8.0 and 7.1 us with 1, 2, 4
  // and 8 ranks; N = 8192, K = 2048: 6.2, 6.4, 6.7 and 11.7.
  const double stage_cost = (kLM + NT) / 144.0 * (C::F4 ? 1.25 : 1.0);
  int splits = 1;
  double best = 0;
  for (int s = 1; s <= 8; s *= 2) {
    const double ctas = (double)tn * tt * s;
    if (s > 1 && (ctas > 2.0 * a.num_sms || chunks < 2 * s)) break;
    const double cost = (chunks + s - 1) / s * stage_cost * std::max(1.0, ctas / a.num_sms) +
                        (s > 1 ? 8 + NT / 8 + (s == 8 ? 2 : 0) : 0);
    if (s == 1 || cost < best) {
      best = cost;
      splits = s;
    }
  }
  // Clusters of 4 and 8 do not fill every SM of a GPC: at one CTA an SM some
  // would wait for a second turn (N = 1024, K = 4096, T = 256: 14 us for 9).
  const int S = splits <= 2 && tn * tt * splits <= a.num_sms ? C::S1 : C::S2;
  auto kern = mx_linear_kernel<XF, WF, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(S));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(tn * splits, tt);
  cfg.blockDim = dim3(kLThreads);
  cfg.dynamicSmemBytes = C::smem(S);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, wmap, xmap, a, splits, S);
}

template <int XF, int WF>
cudaError_t launch_linear_t(const MxLinearArgs& a, cudaStream_t st) {
  // Token tiles of a call start at multiples of 128 (a scale tile's rows) or
  // there is one: the smallest that holds T.  Past 128 tokens these tiles are
  // taken while every SM gets at most one; beyond that the pairs' 256 x 256
  // tiles, with half of the copies, win.  K = 4096, 8x4 bits, N = 4096: 12.0 us
  // here against 13.9 at T = 256; N = 16384: 21.4 against 16.5.
  if (a.T <= 16) return launch_linear<XF, WF, 16>(a, st);
  if (a.T <= 32) return launch_linear<XF, WF, 32>(a, st);
  if (a.T <= 64) return launch_linear<XF, WF, 64>(a, st);
  if (a.T <= 128 || mx_ceil(a.T, 128) * mx_ceil(a.N, kLM) <= a.num_sms)
    return launch_linear<XF, WF, 128>(a, st);
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
