// mx_quant.cu -- rows to microscaled codes and back, and scale planes from
// row order to the product's tiles.
//
// All three are one pass over their data: bound by HBM where that is large
// and by the launch where it is small.  A thread takes groups of 8 elements
// (one 16- or two 16-byte loads), four lanes a block of 32; the block's scale
// comes from two shuffles.  A thread loads its groups, kQThreads apart, before
// it uses the first.  Matrix, row and column of the first come from its flat
// index by division, those of the next by adding: with a division for each the
// kernel was bound by instructions (36 us for 8192 x 4096 bf16 to FP8, 2.8
// TB/s).
#include "mx.cuh"
#include "tc05.cuh"

namespace strata {

namespace {

constexpr int kQThreads = 256;
constexpr int kQUnroll = 4;

// Matrix, row and group of 8 columns of a flat group index, for rows of `per`
// groups and matrices of `rows` rows (padding included).
struct Walk {
  uint32_t per, rows;
  uint32_t step_row, step_c;  // kQThreads = step_row * per + step_c
  uint64_t total;
};
Walk make_walk(int64_t batch, int64_t rows, int64_t per) {
  Walk w;
  w.per = (uint32_t)per;
  w.rows = (uint32_t)rows;
  w.step_row = (uint32_t)(kQThreads / per);
  w.step_c = (uint32_t)(kQThreads % per);
  w.total = (uint64_t)(batch * rows * per);
  return w;
}
struct Place {
  uint32_t batch, row, c;
};
STRATA_DEVFN Place first_place(const Walk& w, uint64_t g) {
  Place p;
  uint32_t r;
  if (w.total >> 32) {
    r = (uint32_t)(g / w.per);
    p.c = (uint32_t)(g - (uint64_t)r * w.per);
  } else {
    r = (uint32_t)g / w.per;
    p.c = (uint32_t)g - r * w.per;
  }
  p.batch = r / w.rows;
  p.row = r - p.batch * w.rows;
  return p;
}
STRATA_DEVFN Place next_place(const Walk& w, Place p) {
  p.c += w.step_c;
  p.row += w.step_row;
  if (p.c >= w.per) {
    p.c -= w.per;
    ++p.row;
  }
  while (p.row >= w.rows) {
    p.row -= w.rows;
    ++p.batch;
  }
  return p;
}

template <int DT, int FMT>
__global__ void __launch_bounds__(kQThreads) mx_quantize_kernel(MxQuantArgs a, Walk w) {
  constexpr int kEl = DT == STRATA_DTYPE_F32 ? 4 : 2;
  const uint32_t groups = (uint32_t)(a.K / 8);
  const int kt = (int)mx_ceil(a.K, kMxTileBlocks * kMxBlock);
  const int64_t row_bytes = mx_row_bytes(FMT, a.K);
  const uint8_t* src = reinterpret_cast<const uint8_t*>(a.src);
  Place p[kQUnroll];
  p[0] = first_place(w, (uint64_t)blockIdx.x * (kQThreads * kQUnroll) + threadIdx.x);
#pragma unroll
  for (int u = 1; u < kQUnroll; ++u) p[u] = next_place(w, p[u - 1]);
  pdl_wait_prior();
  Raw8<DT> raw[kQUnroll];
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    if (p[u].batch < a.batch && p[u].row < a.rows && p[u].c < groups)
      raw[u].load(src + ((int64_t)p[u].batch * a.batch_stride + (int64_t)p[u].row * a.row_stride +
                         (int64_t)p[u].c * 8) * kEl);
    else
      raw[u].zero();  // padding of a scale tile: scale byte 0
  }
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    float v[8];
    raw[u].values(v);
    uint2 codes;
    const uint32_t e = mx_encode8<FMT>(v, raw[u].max_bits(v), codes);
    if (p[u].batch >= a.batch) continue;
    if (p[u].row < a.rows && p[u].c < groups) {
      uint8_t* o = a.codes + p[u].batch * a.codes_stride + (int64_t)p[u].row * row_bytes +
                   mx_row_bytes(FMT, 8) * p[u].c;
      if constexpr (FMT == STRATA_MX_FP4)
        *reinterpret_cast<uint32_t*>(o) = codes.x;
      else
        *reinterpret_cast<uint2*>(o) = codes;
    }
    if ((threadIdx.x & 3) == 0) {
      const int blk = (int)(p[u].c / 4);
      uint8_t* s = a.scales + p[u].batch * a.scales_stride;
      if (a.layout == STRATA_MX_TILES)
        s[mx_tile_byte((int)p[u].row, blk, kt)] = (uint8_t)e;
      else
        s[(int64_t)p[u].row * (groups / 4) + blk] = (uint8_t)e;
    }
  }
}

template <int DT, int FMT>
__global__ void __launch_bounds__(kQThreads) mx_dequantize_kernel(MxDequantArgs a, Walk w) {
  constexpr int kEl = DT == STRATA_DTYPE_F32 ? 4 : 2;
  const int kt = (int)mx_ceil(a.K, kMxTileBlocks * kMxBlock);
  const int64_t row_bytes = mx_row_bytes(FMT, a.K);
  uint8_t* dst = reinterpret_cast<uint8_t*>(a.dst);
  Place p[kQUnroll];
  p[0] = first_place(w, (uint64_t)blockIdx.x * (kQThreads * kQUnroll) + threadIdx.x);
#pragma unroll
  for (int u = 1; u < kQUnroll; ++u) p[u] = next_place(w, p[u - 1]);
  pdl_wait_prior();
  uint2 codes[kQUnroll];
  uint32_t e[kQUnroll];
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    codes[u] = make_uint2(0u, 0u);
    e[u] = 0;
    if (p[u].batch < a.batch) {
      const uint8_t* c = a.codes + p[u].batch * a.codes_stride + (int64_t)p[u].row * row_bytes +
                         mx_row_bytes(FMT, 8) * p[u].c;
      if constexpr (FMT == STRATA_MX_FP4)
        codes[u].x = *reinterpret_cast<const uint32_t*>(c);
      else
        codes[u] = *reinterpret_cast<const uint2*>(c);
      const int blk = (int)(p[u].c / 4);
      const uint8_t* s = a.scales + p[u].batch * a.scales_stride;
      e[u] = a.layout == STRATA_MX_TILES ? s[mx_tile_byte((int)p[u].row, blk, kt)]
                                         : s[(int64_t)p[u].row * (w.per / 4) + blk];
    }
  }
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    if (p[u].batch >= a.batch) continue;
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
  // with tiles, the padding rows and blocks of the scale tiles are visited too
  const bool tiles = a.layout == STRATA_MX_TILES;
  const Walk w = make_walk(a.batch, tiles ? mx_ceil(a.rows, kMxTileRows) * kMxTileRows : a.rows,
                           tiles ? mx_ceil(a.K, 128) * 16 : a.K / 8);
  constexpr uint64_t cta = kQThreads * kQUnroll;
#define STRATA_Q(DT, FMT)                 \
  if (a.src_dtype == DT && a.fmt == FMT)  \
    return launch_groups(mx_quantize_kernel<DT, FMT>, w.total, cta, st, a, w);
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
  const Walk w = make_walk(a.batch, a.rows, a.K / 8);
  constexpr uint64_t cta = kQThreads * kQUnroll;
#define STRATA_D(DT, FMT)                 \
  if (a.dst_dtype == DT && a.fmt == FMT)  \
    return launch_groups(mx_dequantize_kernel<DT, FMT>, w.total, cta, st, a, w);
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
