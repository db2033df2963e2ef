// mx_quant.cu -- rows to microscaled codes and back, and scale planes from
// row order to the product's tiles.
//
// All three are one pass over their data: bound by HBM where that is large
// and by the launch where it is small.  A thread takes 8 elements (one 16- or
// two 16-byte loads), four lanes a block of 32; the block's scale comes from
// two shuffles.  Four groups of 8 a thread are loaded before the first is
// used.  Rows, matrices and padding are found from a flat group index whose
// one 64-bit division is per CTA.
#include "mx.cuh"
#include "tc05.cuh"

namespace strata {

namespace {

constexpr int kQThreads = 256;
constexpr int kQUnroll = 4;

// Where group `i` (of 8 elements) of this CTA's kQThreads * kQUnroll lies:
// rows of `per` groups, matrices of `rows_p` rows.
struct Place {
  uint32_t batch, row, c;
};
STRATA_DEVFN Place place_of(uint64_t row0, uint32_t c0, uint32_t i, uint32_t per,
                            uint32_t rows_p) {
  const uint32_t l = c0 + i, dr = l / per;
  const uint32_t r = (uint32_t)row0 + dr;
  Place p;
  p.c = l - dr * per;
  p.batch = r / rows_p;
  p.row = r - p.batch * rows_p;
  return p;
}

template <int DT, int FMT>
__global__ void __launch_bounds__(kQThreads) mx_quantize_kernel(MxQuantArgs a, uint32_t per,
                                                                uint32_t rows_p, uint64_t total) {
  constexpr int kEl = DT == STRATA_DTYPE_F32 ? 4 : 2;
  const uint64_t g0 = (uint64_t)blockIdx.x * (kQThreads * kQUnroll);
  const uint64_t row0 = g0 / per;
  const uint32_t c0 = (uint32_t)(g0 - row0 * per);
  const uint32_t groups = (uint32_t)(a.K / 8);
  const int kt = (int)mx_ceil(a.K, kMxTileBlocks * kMxBlock);
  const uint8_t* src = reinterpret_cast<const uint8_t*>(a.src);
  pdl_wait_prior();
  float v[kQUnroll][8];
  Place p[kQUnroll];
  bool in[kQUnroll], live[kQUnroll];
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    const uint32_t i = u * kQThreads + threadIdx.x;
    in[u] = g0 + i < total;
    p[u] = place_of(row0, c0, i, per, rows_p);
    live[u] = in[u] && p[u].row < (uint32_t)a.rows && p[u].c < groups;
    if (live[u]) {
      load8<DT>(src + ((int64_t)p[u].batch * a.batch_stride + (int64_t)p[u].row * a.row_stride +
                       (int64_t)p[u].c * 8) * kEl,
                v[u]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = 0.f;  // padding of a scale tile: scale byte 0
    }
  }
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    uint2 codes;
    const uint32_t e = mx_encode8<FMT>(v[u], codes);
    if (live[u]) {
      uint8_t* o = a.codes + p[u].batch * a.codes_stride +
                   (int64_t)p[u].row * mx_row_bytes(FMT, a.K) + mx_row_bytes(FMT, 8) * p[u].c;
      if constexpr (FMT == STRATA_MX_FP4)
        *reinterpret_cast<uint32_t*>(o) = codes.x;
      else
        *reinterpret_cast<uint2*>(o) = codes;
    }
    if (in[u] && (threadIdx.x & 3) == 0) {
      const int blk = (int)(p[u].c / 4);
      uint8_t* s = a.scales + p[u].batch * a.scales_stride;
      if (a.layout == STRATA_MX_TILES)
        s[mx_tile_byte((int)p[u].row, blk, kt)] = (uint8_t)e;
      else
        s[(int64_t)p[u].row * (a.K / kMxBlock) + blk] = (uint8_t)e;
    }
  }
}

template <int DT, int FMT>
__global__ void __launch_bounds__(kQThreads) mx_dequantize_kernel(MxDequantArgs a, uint32_t per,
                                                                  uint64_t total) {
  constexpr int kEl = DT == STRATA_DTYPE_F32 ? 4 : 2;
  const uint64_t g0 = (uint64_t)blockIdx.x * (kQThreads * kQUnroll);
  const uint64_t row0 = g0 / per;
  const uint32_t c0 = (uint32_t)(g0 - row0 * per);
  const int kt = (int)mx_ceil(a.K, kMxTileBlocks * kMxBlock);
  uint8_t* dst = reinterpret_cast<uint8_t*>(a.dst);
  pdl_wait_prior();
  uint2 codes[kQUnroll];
  uint32_t e[kQUnroll];
  Place p[kQUnroll];
  bool in[kQUnroll];
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    const uint32_t i = u * kQThreads + threadIdx.x;
    in[u] = g0 + i < total;
    p[u] = place_of(row0, c0, i, per, (uint32_t)a.rows);
    codes[u] = make_uint2(0u, 0u);
    e[u] = 0;
    if (in[u]) {
      const uint8_t* c = a.codes + p[u].batch * a.codes_stride +
                         (int64_t)p[u].row * mx_row_bytes(FMT, a.K) + mx_row_bytes(FMT, 8) * p[u].c;
      if constexpr (FMT == STRATA_MX_FP4)
        codes[u].x = *reinterpret_cast<const uint32_t*>(c);
      else
        codes[u] = *reinterpret_cast<const uint2*>(c);
      const int blk = (int)(p[u].c / 4);
      const uint8_t* s = a.scales + p[u].batch * a.scales_stride;
      e[u] = a.layout == STRATA_MX_TILES ? s[mx_tile_byte((int)p[u].row, blk, kt)]
                                         : s[(int64_t)p[u].row * (a.K / kMxBlock) + blk];
    }
  }
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    if (!in[u]) continue;
    float v[8];
    mx_decode8<FMT>(codes[u], e[u], v);
    store8<DT>(dst + ((int64_t)p[u].batch * a.batch_stride + (int64_t)p[u].row * a.row_stride +
                      (int64_t)p[u].c * 8) * kEl,
               v);
  }
}

// One thread a 4-byte word of a tile: a row's four blocks.
__global__ void __launch_bounds__(kQThreads) mx_tile_scales_kernel(const uint8_t* __restrict__ src,
                                                                   int64_t rows, int nb, int kt,
                                                                   uint64_t words,
                                                                   uint32_t* __restrict__ dst) {
  pdl_wait_prior();
  const uint64_t w = (uint64_t)blockIdx.x * kQThreads + threadIdx.x;
  if (w >= words) return;
  const uint64_t tile = w / (kMxTileBytes / 4);
  const uint32_t in = (uint32_t)(w % (kMxTileBytes / 4));  // lane * 4 + row group
  const int64_t row = (int64_t)(tile / kt) * kMxTileRows + (in % 4) * 32 + in / 4;
  const int b0 = (int)(tile % kt) * kMxTileBlocks;
  uint32_t v = 0;
  if (row < rows) {
    for (int i = 0; i < kMxTileBlocks; ++i)
      if (b0 + i < nb) v |= (uint32_t)src[row * nb + b0 + i] << (8 * i);
  }
  dst[w] = v;
}

template <typename Kern, typename... A>
cudaError_t launch_groups(Kern kern, uint64_t total, uint64_t per_cta, cudaStream_t st,
                          A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)((total + per_cta - 1) / per_cta));
  cfg.blockDim = dim3(kQThreads);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantArgs& a, cudaStream_t st) {
  const bool tiles = a.layout == STRATA_MX_TILES;
  // with tiles, the padding rows and blocks of the scale tiles are visited too
  const uint32_t per = (uint32_t)(tiles ? mx_ceil(a.K, 128) * 16 : a.K / 8);
  const uint32_t rows_p =
      (uint32_t)(tiles ? mx_ceil(a.rows, kMxTileRows) * kMxTileRows : a.rows);
  const uint64_t total = (uint64_t)a.batch * rows_p * per;
  constexpr uint64_t cta = kQThreads * kQUnroll;
#define STRATA_Q(DT, FMT)                                                                     \
  if (a.src_dtype == DT && a.fmt == FMT)                                                      \
    return launch_groups(mx_quantize_kernel<DT, FMT>, total, cta, st, a, per, rows_p, total);
  STRATA_Q(STRATA_DTYPE_F32, STRATA_MX_FP4)
  STRATA_Q(STRATA_DTYPE_F16, STRATA_MX_FP4)
  STRATA_Q(STRATA_DTYPE_BF16, STRATA_MX_FP4)
  STRATA_Q(STRATA_DTYPE_F32, STRATA_MX_FP8)
  STRATA_Q(STRATA_DTYPE_F16, STRATA_MX_FP8)
  STRATA_Q(STRATA_DTYPE_BF16, STRATA_MX_FP8)
#undef STRATA_Q
  return cudaErrorInvalidValue;
}

cudaError_t launch_mx_dequantize(const MxDequantArgs& a, cudaStream_t st) {
  const uint32_t per = (uint32_t)(a.K / 8);
  const uint64_t total = (uint64_t)a.batch * a.rows * per;
  constexpr uint64_t cta = kQThreads * kQUnroll;
#define STRATA_D(DT, FMT)                                                                \
  if (a.dst_dtype == DT && a.fmt == FMT)                                                 \
    return launch_groups(mx_dequantize_kernel<DT, FMT>, total, cta, st, a, per, total);
  STRATA_D(STRATA_DTYPE_F32, STRATA_MX_FP4)
  STRATA_D(STRATA_DTYPE_F16, STRATA_MX_FP4)
  STRATA_D(STRATA_DTYPE_BF16, STRATA_MX_FP4)
  STRATA_D(STRATA_DTYPE_F32, STRATA_MX_FP8)
  STRATA_D(STRATA_DTYPE_F16, STRATA_MX_FP8)
  STRATA_D(STRATA_DTYPE_BF16, STRATA_MX_FP8)
#undef STRATA_D
  return cudaErrorInvalidValue;
}

cudaError_t launch_mx_tile_scales(const uint8_t* src, int64_t rows, int64_t K, uint8_t* dst,
                                  cudaStream_t st) {
  const uint64_t words = (uint64_t)mx_scale_plane(rows, K, STRATA_MX_TILES) / 4;
  return launch_groups(mx_tile_scales_kernel, words, (uint64_t)kQThreads, st, src, rows,
                       (int)(K / kMxBlock), (int)mx_ceil(K, 128), words,
                       reinterpret_cast<uint32_t*>(dst));
}

}  // namespace strata
