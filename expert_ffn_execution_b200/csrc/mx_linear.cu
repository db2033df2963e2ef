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
// x NT tokens; where there are fewer tiles than SMs the K axis is split over a
// cluster of up to 8 CTAs, and every CTA joins the sums of some of the tokens
// in rank order.  Joining is a matter of round trips: with T = 4, N = 2560, K =
// 2560, 8x4 bits, fetching the sums 16 bytes at a time behind a barrier that
// orders memory took 5.2 us, and 4.5 us once each CTA sent a rank its tokens
// by one bulk copy that counts on the receiver's barrier (3.9 us now).
#include <algorithm>

#include "deal.h"
#include "mx_mma.cuh"
#include "mx_plan.h"
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
  static constexpr int sfcols = 8 * ST;  // tensor-memory columns of a stage's scales
  static constexpr int dcols = NT < 32 ? 32 : NT;
  static constexpr int head = 1024;      // barriers, and the alignment of what follows
  static constexpr int token = kLM * 4;  // bytes of a token's sums
  // Stages of a CTA with `room` bytes; a split K also takes the sums that are
  // sent to it.
  static constexpr int stages(int room, bool split) {
    return (room - head - 1024 - (split ? NT * token : 0)) / stride;
  }
  static constexpr int kAlone = 227 * 1024, kShared = 113 * 1024;  // one CTA an SM, two
  static constexpr int smem(int S, bool split) {
    return S * stride + head + 1024 + (split ? NT * token : 0);
  }
  // The most that any call of the kernel asks for.  What a kernel may ask for is
  // the process's, not the call's: set to less for one call, it would be too
  // little for another thread's.
  static constexpr int kMost =
      std::max(std::max(smem(stages(kAlone, false), false), smem(stages(kAlone, true), true)),
               std::max(smem(stages(kShared, false), false), smem(stages(kShared, true), true)));
  static_assert(kMost <= 227 * 1024, "what an SM has for a CTA");
  static constexpr int cols(int S) {
    return dcols + S * sfcols <= 64 ? 64 : dcols + S * sfcols <= 128 ? 128 : 256;
  }
  static_assert(dcols + stages(kAlone, false) * sfcols <= 256, "at most half of the tensor memory");
  static_assert(stages(kShared, false) * stride >= NT * token, "the sums fit over the stages");
  static_assert(NT == 128 || (stages(kShared, true) * stride >= NT * token &&
                              stages(kShared, true) >= 3), "and with a split K");
  static_assert((2 * stages(kAlone, false) + 2) * 8 + 16 <= head, "the barriers fit");
};

template <int DT>
STRATA_DEVFN void store1(void* y, int64_t i, float v) {
  if constexpr (DT == STRATA_DTYPE_F32)
    reinterpret_cast<float*>(y)[i] = v;
  else
    reinterpret_cast<uint16_t*>(y)[i] = (uint16_t)pack2<DT>(v, v);
}
template <int N>  // N columns of this warp's 32 lanes
STRATA_DEVFN void tmem_load(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 32, "what a tile has");
  if constexpr (N == 16)
    tmem_ld16(taddr, r);
  else
    tmem_ld32(taddr, r);
  tmem_wait_ld();
}
// The sums of this warp's 32 features and `count` tokens in tensor memory -> y,
// element i on for the lane's feature (`some`: it is one of y's).  A lane has a
// feature and its tokens are registers, so a token's store is 32 elements side
// by side, on any alignment, and takes few instructions: through shared memory
// and by wider stores 64 tokens took 4900 cycles after the last MMA, of code
// that runs once.
template <int DT, int NT>
STRATA_DEVFN void write_sums(const MxLinearArgs& a, uint32_t taddr, int64_t i, bool some,
                             float bias, int count) {
  constexpr int kLoad = NT < 32 ? 16 : 32;
#pragma unroll 1
  for (int c = 0; c < count; c += kLoad) {
    uint32_t r[kLoad];
    tmem_load<kLoad>(taddr + c, r);
#pragma unroll
    for (int k = 0; k < kLoad; ++k, i += a.ldy)
      if (some && c + k < count) store1<DT>(a.y, i, __uint_as_float(r[k]) + bias);
  }
}
// Sums [rank][token][feature], ranks `per` tokens apart, of `count` tokens, rank
// by rank -> y, element i on for this thread's feature.
template <int DT, int SPLITS>
STRATA_DEVFN void write_joined(const MxLinearArgs& a, const float* sums, int64_t i, float bias,
                               int count, int per) {
#pragma unroll 2
  for (int t = 0; t < count; ++t, i += a.ldy, sums += kLM) {
    float v[SPLITS];
#pragma unroll
    for (int q = 0; q < SPLITS; ++q) v[q] = sums[q * per * kLM];
#pragma unroll
    for (int q = 1; q < SPLITS; ++q) v[0] += v[q];
    store1<DT>(a.y, i, v[0] + bias);
  }
}
template <int DT>
STRATA_DEVFN void write_joined(const MxLinearArgs& a, const float* sums, int64_t i, float bias,
                               int count, int per, int splits) {
  if (splits == 2) write_joined<DT, 2>(a, sums, i, bias, count, per);
  if (splits == 4) write_joined<DT, 4>(a, sums, i, bias, count, per);
  if (splits == 8) write_joined<DT, 8>(a, sums, i, bias, count, per);
}

template <int XF, int WF, int NT>
__global__ void __launch_bounds__(kLThreads)
mx_linear_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
                 MxLinearArgs a, int lg_splits, int S) {
  using C = LinCfg<XF, WF, NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem0 =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* smem = smem0 + C::head;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem0);
  uint64_t* empty = full + S;
  uint64_t* tfull = empty + S;
  uint64_t* joined = tfull + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(joined + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* issued = reinterpret_cast<int*>(tmem_slot + 2);

  // the warp from one lane: known to be the same in all, as is what follows from it
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
  // (shifts: divisions here took 0.3 us before the first barrier)
  const int splits = 1 << lg_splits;
  const int rank = splits > 1 ? (int)cluster_ctarank() : 0;
  const int n0 = (int)(blockIdx.x >> lg_splits) * kLM, t0 = blockIdx.y * NT;
  const int kt = a.K / 128;                          // scale tiles of a row block
  const int chunks = (a.K + C::KS - 1) / C::KS;
  const int c0 = chunks * rank >> lg_splits;
  const int nch = (chunks * (rank + 1) >> lg_splits) - c0;

  // the tile's tokens, and those that this rank joins: [rank per, rank per + mine)
  const int nt = min(NT, a.T - t0), per = (nt + splits - 1) >> lg_splits;
  const int first = rank * per, mine = max(0, min(per, nt - first));
  if ((int)threadIdx.x < 2 * S + 2) {  // one barrier a thread: in turn they took 0.4 us
    mbar_init(&full[threadIdx.x], 1);
    fence_barrier_init();
  }
  if (threadIdx.x == kLThreads - 1) {
    *abort_flag = 0;
    *issued = 0;
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
  const uint32_t tbase = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  if (splits > 1) {
    if (threadIdx.x == 0)  // every rank sends this one its sums of `mine` tokens
      mbar_arrive_expect_tx(joined, (uint32_t)(mine * splits * C::token));
    __syncwarp();
    cluster_arrive_relaxed();  // waited for before the first copy to another rank
  }
  const int n = n0 + (int)threadIdx.x;  // the feature of a thread that reads sums
  const bool some = (int)threadIdx.x < kLM && n < a.N;
  float bias = 0.f;
  pdl_wait_prior();

  if (warp == 4) {
    int i = 0, s = 0;
    uint32_t ph = 1;
    for (; i < nch; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait_guarded(&empty[s], ph, a.status, abort_flag))) break;
      const int ch = c0 + i;
      const uint32_t scales = (uint32_t)min(C::ST, kt - ch * C::ST) * kMxTileBytes;  // left along K
      uint8_t* st = smem + s * C::stride;
      // coordinates in the map's elements: codes of the spread type, else bytes
      const int kw = C::kSpread ? ch * C::KS : (int)mx_row_bytes(WF, (int64_t)ch * C::KS);
      const int kx = (int)mx_row_bytes(XF, (int64_t)ch * C::KS);
      load_stage_warp(&full[s], C::WTx + C::XB + 2 * scales, &wmap, kw, n0, st, &xmap, kx, t0,
                      st + C::WB,
                      a.w_scales + ((int64_t)(n0 / 128) * kt + ch * C::ST) * kMxTileBytes,
                      st + C::WB + C::XB,
                      a.x_scales + ((int64_t)(t0 / 128) * kt + ch * C::ST) * kMxTileBytes,
                      st + C::WB + C::XB + C::SB, scales);
      if (++s == S) s = 0, ph ^= 1u;
    }
    *issued = i;
    __syncwarp();
  } else if (warp == 5) {
    const uint32_t hi = smem_desc_k128_hi(1024);
    const uint32_t stages = smem_addr(smem);
    constexpr uint32_t wf = C::F4 ? 1u : WF == STRATA_MX_FP4 ? 5u : 0u;
    constexpr uint32_t xf = C::F4 ? 1u : XF == STRATA_MX_FP4 ? 5u : 0u;
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < nch; ++i) {
      if (!__all_sync(0xffffffffu, mbar_wait_guarded(&full[s], ph, a.status, abort_flag))) break;
      tc_fence_after();
      const int left = a.K - (c0 + i) * C::KS;  // a multiple of 128
      const uint32_t st = stages + (uint32_t)(s * C::stride);
      // a tile that starts 64 tokens into its scale tile reads two columns on
      const uint32_t sfw = tbase + C::dcols + s * C::sfcols, sfx = sfw + 4 * C::ST;
      const uint32_t sfx_at = sfx + (NT == 64 ? (t0 % 128) / 32 : 0);
      const uint32_t wlo = smem_desc_k128_lo(st), xlo = smem_desc_k128_lo(st + C::WB);
#pragma unroll
      for (int b = 0; b < C::ST; ++b) {
        if (b * 128 < left) {
          const uint32_t scales = st + C::WB + C::XB + b * kMxTileBytes;
          mma_mx_block<C::F4, false>(
              tbase, wlo + 4 * b, xlo + 4 * b, hi, idesc_mx(wf, xf, kLM, NT, 0), sfw + 4 * b,
              sfx + 4 * b, sfx_at + 4 * b, smem_desc_scale_lo(scales),
              smem_desc_scale_lo(scales + C::SB), 0u, (uint32_t)(i + b > 0));
        }
      }
      mma_commit_warp(&empty[s]);
      if (++s == S) s = 0, ph ^= 1u;
    }
    mma_commit_warp(tfull);
    __syncwarp();
  } else {
    if (some && a.bias) bias = a.bias[n];
    const bool ok = __all_sync(0xffffffffu, mbar_wait_guarded(tfull, 0, a.status, abort_flag) &&
                                                !*abort_flag);
    tc_fence_after();
    const uint32_t tq = tbase + ((uint32_t)(warp * 32) << 16);
    if (ok && splits == 1) {
      const int64_t y0 = (int64_t)t0 * a.ldy + n;
      if (a.y_dtype == STRATA_DTYPE_F32)
        write_sums<STRATA_DTYPE_F32, NT>(a, tq, y0, some, bias, nt);
      else if (a.y_dtype == STRATA_DTYPE_F16)
        write_sums<STRATA_DTYPE_F16, NT>(a, tq, y0, some, bias, nt);
      else
        write_sums<STRATA_DTYPE_BF16, NT>(a, tq, y0, some, bias, nt);
    } else if (ok) {
      // sums -> shared memory [token][feature], over the stages
      constexpr int kLoad = NT < 32 ? 16 : 32;
      float* red = reinterpret_cast<float*>(smem) + threadIdx.x;
#pragma unroll 1
      for (int c = 0; c < nt; c += kLoad) {
        uint32_t r[kLoad];
        tmem_load<kLoad>(tq + c, r);
#pragma unroll
        for (int i = 0; i < kLoad; ++i) red[(c + i) * kLM] = __uint_as_float(r[i]);
      }
    }
    if (splits > 1) fence_proxy_async_smem();  // read by the bulk copies
    tc_fence_before();
  }
  __syncthreads();
  if (*abort_flag) {  // the same for all threads: every guarded wait is behind them
    // a wait gave up: every copy that was started lands, and every MMA ends,
    // before the shared and tensor memory are released (bounded)
    if (threadIdx.x == 0) {
      const int started = *issued;
      for (int s = 0; s < S && s < started; ++s)
        mbar_wait_bounded(&full[s], last_armed_parity(started, S, s), a.status, kLDrainCycles);
      mbar_wait_bounded(tfull, 0, a.status, kLDrainCycles);
    }
    __syncthreads();
  }
  // Tensor memory goes before the other ranks are waited for: a rank that is
  // itself waiting for tensor memory (another kernel's CTA has it) holds none.
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tbase, C::cols(S));
  }
  __syncwarp();
  if (splits > 1) {
    cluster_wait();
    const uint8_t* sums = smem + S * C::stride;
    if ((int)threadIdx.x < splits) {
      const int to = threadIdx.x, count = min(per, nt - to * per);
      if (count > 0)
        bulk_s2cluster(cluster_addr(smem_addr(sums) + rank * per * C::token, to),
                       smem_addr(smem) + to * per * C::token, (uint32_t)(count * C::token),
                       cluster_addr(smem_addr(joined), to));
    }
    __syncwarp();
    // not guarded by the abort flag: every rank sends, and what is on its way
    // here has to land before this CTA goes
    if (mbar_wait_bounded(joined, 0, a.status) && some) {
      const float* at = reinterpret_cast<const float*>(sums) + threadIdx.x;
      const int64_t y0 = (int64_t)(t0 + first) * a.ldy + n;
      if (a.y_dtype == STRATA_DTYPE_F32)
        write_joined<STRATA_DTYPE_F32>(a, at, y0, bias, mine, per, splits);
      else if (a.y_dtype == STRATA_DTYPE_F16)
        write_joined<STRATA_DTYPE_F16>(a, at, y0, bias, mine, per, splits);
      else
        write_joined<STRATA_DTYPE_BF16>(a, at, y0, bias, mine, per, splits);
    }
    __syncwarp();
    // nobody leaves while its sums are being sent
    cluster_sync_relaxed();
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
cudaError_t launch_linear(const MxLinearArgs& a, int splits, cudaStream_t st) {
  using C = LinCfg<XF, WF, NT>;
  CUtensorMap wmap, xmap;
  if (!make_mx_map(&wmap, a.w_codes, WF, C::kSpread, a.N, a.K, kLM) ||
      !make_mx_map(&xmap, a.x_codes, XF, false, a.T, a.K, NT))
    return cudaErrorInvalidValue;
  const int tn = (a.N + kLM - 1) / kLM, tt = (a.T + NT - 1) / NT;
  const bool split = splits > 1;
  const int lg = splits == 8 ? 3 : splits == 4 ? 2 : splits == 2 ? 1 : 0;
  // Clusters of 4 and 8 do not fill every SM of a GPC: at one CTA an SM some
  // would wait for a second turn (T = 4, N = 2304, K = 8192, 8 ranks: 10.2 us
  // for 6.4).
  const bool alone = splits <= 2 && (int64_t)tn * tt * splits <= a.num_sms;
  const int S = C::stages(alone ? C::kAlone : C::kShared, split);
  auto kern = mx_linear_kernel<XF, WF, NT>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kMost);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(tn * splits, tt);
  cfg.blockDim = dim3(kLThreads);
  cfg.dynamicSmemBytes = C::smem(S, split);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, wmap, xmap, a, lg, S);
}

template <int XF, int WF>
cudaError_t launch_linear_t(const MxLinearArgs& a, cudaStream_t st) {
  const LinPlan p = plan_linear(a.T, a.N, a.K, XF == STRATA_MX_FP4 && WF == STRATA_MX_FP4, a.num_sms);
  switch (p.nt) {
    case 0: return launch_mx_gemm(a, st);
    case 16: return launch_linear<XF, WF, 16>(a, p.splits, st);
    case 32: return launch_linear<XF, WF, 32>(a, p.splits, st);
    case 64: return launch_linear<XF, WF, 64>(a, p.splits, st);
    default: return launch_linear<XF, WF, 128>(a, p.splits, st);
  }
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
