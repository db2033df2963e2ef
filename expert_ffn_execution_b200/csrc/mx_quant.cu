// mx_quant.cu -- rows to microscaled codes and back, and scale planes from
// row order to the product's tiles.
//
// All three are one pass over their data: bound by HBM where that is large
// and by the launch where it is small; in between, by instructions, so what is
// not the conversion itself is kept small.  A thread takes 16 elements at a
// time (half a block: one shuffle joins two lanes' largest magnitudes), and
// loads its kQUnroll pieces, kQThreads apart, before it uses the first (32
// experts of 2560 x 640 to MXFP4: 83, 72 and 78 us with 1, 2 and 4).
// Matrix, row and column of the first come from its flat index by division,
// those of the next, and their offsets, by adding.  8192 x 4096 bf16 to FP8:
// 36 us with 8 elements and three divisions a piece, 24 us without the
// divisions, 18 us with 16 elements and added offsets, 17 us (6.0 TB/s) with
// products two an instruction and tile offsets in unsigned arithmetic.
#include "mx.cuh"
#include "tc05.cuh"

namespace strata {

namespace {

constexpr int kQThreads = 256;
constexpr int kQUnroll = 2;
constexpr int kQEl = 16;  // elements of a piece

// A walk over the pieces of a batch of matrices, kQThreads at a step, for rows
// of `per` pieces and matrices of `rows` rows (padding included).
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
// An offset linear in matrix, row and piece: what a step, the end of a row
// and the end of a matrix add.
struct Stride {
  int64_t batch, row, piece;
  int64_t step, row_end, batch_end;
};
Stride make_stride(const Walk& w, int64_t batch, int64_t row, int64_t piece) {
  Stride s;
  s.batch = batch;
  s.row = row;
  s.piece = piece;
  s.step = (int64_t)w.step_row * row + (int64_t)w.step_c * piece;
  s.row_end = row - (int64_t)w.per * piece;
  s.batch_end = batch - (int64_t)w.rows * row;
  return s;
}
struct Place {
  uint32_t batch, row, c;
  int64_t src, dst;  // offsets by the two strides
};
STRATA_DEVFN Place first_place(const Walk& w, const Stride& src, const Stride& dst, uint64_t g) {
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
  p.src = p.batch * src.batch + p.row * src.row + p.c * src.piece;
  p.dst = p.batch * dst.batch + p.row * dst.row + p.c * dst.piece;
  return p;
}
STRATA_DEVFN Place next_place(const Walk& w, const Stride& src, const Stride& dst, Place p) {
  p.c += w.step_c;
  p.row += w.step_row;
  p.src += src.step;
  p.dst += dst.step;
  if (p.c >= w.per) {
    p.c -= w.per;
    ++p.row;
    p.src += src.row_end;
    p.dst += dst.row_end;
  }
  while (p.row >= w.rows) {
    p.row -= w.rows;
    ++p.batch;
    p.src += src.batch_end;
    p.dst += dst.batch_end;
  }
  return p;
}
// The scale byte of a place's block.
STRATA_DEVFN int64_t scale_at(const Place& p, int layout, uint64_t batch_stride, int64_t blocks,
                              int kt) {
  const int blk = (int)(p.c / 2);
  return (int64_t)(p.batch * batch_stride) +
         (layout == STRATA_MX_TILES ? mx_tile_byte((int)p.row, blk, kt) : p.row * blocks + blk);
}

// Up to three batches a launch (the planes of expert blobs), one after the
// other over the grid: batch i has blocks first[i] .. first[i + 1] - 1.
template <typename Args>
struct Jobs {
  Args a[3];
  Walk w[3];
  Stride src[3], dst[3];
  uint32_t first[4];
};
// MANY: more than one batch.  One alone is known at compile time (52M bf16 to
// MXFP4: 24.2 us for 25.7).
template <bool MANY, typename Args>
STRATA_DEVFN int job_of(const Jobs<Args>& j) {
  return MANY ? (blockIdx.x >= j.first[1]) + (blockIdx.x >= j.first[2]) : 0;
}
// The places of this thread's pieces.
template <typename Args>
STRATA_DEVFN void places_of(const Jobs<Args>& jobs, int j, Place (&p)[kQUnroll]) {
  const Walk& w = jobs.w[j];
  const uint64_t block = blockIdx.x - jobs.first[j];
  p[0] = first_place(w, jobs.src[j], jobs.dst[j], block * (kQThreads * kQUnroll) + threadIdx.x);
#pragma unroll
  for (int u = 1; u < kQUnroll; ++u) p[u] = next_place(w, jobs.src[j], jobs.dst[j], p[u - 1]);
}

template <int DT, int FMT, bool MANY>
__global__ void __launch_bounds__(kQThreads)
mx_quantize_kernel(const __grid_constant__ Jobs<MxQuantArgs> jobs) {
  const int j = job_of<MANY>(jobs);
  const MxQuantArgs& a = jobs.a[j];
  const uint32_t pieces = (uint32_t)(a.K / kQEl);
  const int kt = (int)mx_ceil(a.K, kMxTileBlocks * kMxBlock);
  const uint8_t* src = reinterpret_cast<const uint8_t*>(a.src);
  Place p[kQUnroll];
  places_of(jobs, j, p);
  pdl_wait_prior();
  // Scales in tiles are the product's operand: its CTAs set up while this grid
  // runs and wait for its end before they read (T = 1, N = 10240, K = 2560,
  // 8x4 bits, quantised and multiplied: 8.9 us without, 8.2 us).  Experts'
  // blobs may be read before a wait: nothing is released for them.
  if (a.layout == STRATA_MX_TILES) pdl_trigger();
  Raw8<DT> raw[kQUnroll][2];
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    if (p[u].batch < a.batch && p[u].row < a.rows && p[u].c < pieces) {
      raw[u][0].load(src + p[u].src);
      raw[u][1].load(src + p[u].src + sizeof(raw[u][0]));
    } else {  // padding of a scale tile: scale byte 0
      raw[u][0].zero();
      raw[u][1].zero();
    }
  }
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    float v0[8], v1[8];
    raw[u][0].values(v0);
    raw[u][1].values(v1);
    uint32_t m = max(raw[u][0].max_bits(v0), raw[u][1].max_bits(v1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t e = mx_scale_of<FMT>(m);
    if (p[u].batch >= a.batch) continue;
    if (p[u].row < a.rows && p[u].c < pieces) {
      const uint2 c0 = mx_encode8<FMT>(v0, e), c1 = mx_encode8<FMT>(v1, e);
      if constexpr (FMT == STRATA_MX_FP4)
        *reinterpret_cast<uint2*>(a.codes + p[u].dst) = make_uint2(c0.x, c1.x);
      else
        *reinterpret_cast<uint4*>(a.codes + p[u].dst) = make_uint4(c0.x, c0.y, c1.x, c1.y);
    }
    if ((threadIdx.x & 1) == 0)
      a.scales[scale_at(p[u], a.layout, a.scales_stride, pieces / 2, kt)] = (uint8_t)e;
  }
}

template <int DT, int FMT, bool MANY>
__global__ void __launch_bounds__(kQThreads)
mx_dequantize_kernel(const __grid_constant__ Jobs<MxDequantArgs> jobs) {
  constexpr int kEl = DT == STRATA_DTYPE_F32 ? 4 : 2;
  const int j = job_of<MANY>(jobs);
  const MxDequantArgs& a = jobs.a[j];
  const int kt = (int)mx_ceil(a.K, kMxTileBlocks * kMxBlock);
  uint8_t* dst = reinterpret_cast<uint8_t*>(a.dst);
  Place p[kQUnroll];
  places_of(jobs, j, p);
  pdl_wait_prior();
  uint2 c0[kQUnroll], c1[kQUnroll];
  uint32_t e[kQUnroll];
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    c0[u] = c1[u] = make_uint2(0u, 0u);
    e[u] = 0;
    if (p[u].batch >= a.batch) continue;
    if constexpr (FMT == STRATA_MX_FP4) {
      const uint2 c = *reinterpret_cast<const uint2*>(a.codes + p[u].src);
      c0[u] = make_uint2(c.x, 0u);
      c1[u] = make_uint2(c.y, 0u);
    } else {
      const uint4 c = *reinterpret_cast<const uint4*>(a.codes + p[u].src);
      c0[u] = make_uint2(c.x, c.y);
      c1[u] = make_uint2(c.z, c.w);
    }
    e[u] = a.scales[scale_at(p[u], a.layout, a.scales_stride, jobs.w[j].per / 2, kt)];
  }
  // The two lanes of a block trade halves of their codes, so that both write
  // the first lane's 16 elements side by side, then the second's: with 16
  // elements a lane in turn every store left half of each 32-byte sector to
  // the next (29 us for 52M MXFP4 values to bf16, against 21.4 us).
  const bool odd = threadIdx.x & 1;
#pragma unroll
  for (int u = 0; u < kQUnroll; ++u) {
    const uint2 give = odd ? c0[u] : c1[u];
    uint2 got;
    got.x = __shfl_xor_sync(0xffffffffu, give.x, 1);
    got.y = FMT == STRATA_MX_FP4 ? 0u : __shfl_xor_sync(0xffffffffu, give.y, 1);
    if (p[u].batch >= a.batch) continue;
    uint8_t* at = dst + p[u].dst - (odd ? 8 * kEl : 0);
    float v[8];
    mx_decode8<FMT>(odd ? got : c0[u], e[u], v);
    store8<DT>(at, v);
    mx_decode8<FMT>(odd ? c1[u] : got, e[u], v);
    store8<DT>(at + kQEl * kEl, v);
  }
}

// One thread a 4-byte word of a tile: a row's four blocks.  A gather of bytes at
// 0.4 to 0.6 TB/s (16384 x 4096: 9.5 us), for a matrix once when it is loaded.
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
cudaError_t launch_blocks(Kern kern, uint64_t blocks, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kQThreads);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Fills in where each job's blocks are; false where the grid would be too large.
template <typename Args>
bool deal_blocks(Jobs<Args>& j, int n) {
  uint64_t at = 0;
  for (int i = 0; i < 4; ++i) {
    j.first[i] = (uint32_t)at;
    if (i < n) at += (uint64_t)mx_ceil((int64_t)j.w[i].total, kQThreads * kQUnroll);
    if (at >= (uint64_t)1 << 31) return false;
  }
  return true;
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantArgs* a, int n, cudaStream_t st) {
  Jobs<MxQuantArgs> j = {};
  for (int i = 0; i < n; ++i) {
    // with tiles, the padding rows and blocks of the scale tiles are visited too
    const bool tiles = a[i].layout == STRATA_MX_TILES;
    const int64_t el = a[i].src_dtype == STRATA_DTYPE_F32 ? 4 : 2;
    j.a[i] = a[i];
    j.w[i] = make_walk(a[i].batch, tiles ? mx_ceil(a[i].rows, kMxTileRows) * kMxTileRows : a[i].rows,
                       tiles ? mx_ceil(a[i].K, 128) * (128 / kQEl) : a[i].K / kQEl);
    j.src[i] = make_stride(j.w[i], a[i].batch_stride * el, a[i].row_stride * el, kQEl * el);
    j.dst[i] = make_stride(j.w[i], (int64_t)a[i].codes_stride, mx_row_bytes(a[i].fmt, a[i].K),
                           mx_row_bytes(a[i].fmt, kQEl));
  }
  if (!deal_blocks(j, n)) return cudaErrorInvalidValue;
#define STRATA_Q(DT, FMT)                     \
  if (a->src_dtype == DT && a->fmt == FMT)    \
    return n > 1 ? launch_blocks(mx_quantize_kernel<DT, FMT, true>, j.first[3], st, j)      \
                 : launch_blocks(mx_quantize_kernel<DT, FMT, false>, j.first[3], st, j);
  STRATA_Q(STRATA_DTYPE_F32, STRATA_MX_FP4)
  STRATA_Q(STRATA_DTYPE_F16, STRATA_MX_FP4)
  STRATA_Q(STRATA_DTYPE_BF16, STRATA_MX_FP4)
  STRATA_Q(STRATA_DTYPE_F32, STRATA_MX_FP8)
  STRATA_Q(STRATA_DTYPE_F16, STRATA_MX_FP8)
  STRATA_Q(STRATA_DTYPE_BF16, STRATA_MX_FP8)
#undef STRATA_Q
  return cudaErrorInvalidValue;
}

cudaError_t launch_mx_dequantize(const MxDequantArgs* a, int n, cudaStream_t st) {
  Jobs<MxDequantArgs> j = {};
  for (int i = 0; i < n; ++i) {
    const int64_t el = a[i].dst_dtype == STRATA_DTYPE_F32 ? 4 : 2;
    j.a[i] = a[i];
    j.w[i] = make_walk(a[i].batch, a[i].rows, a[i].K / kQEl);
    j.src[i] = make_stride(j.w[i], (int64_t)a[i].codes_stride, mx_row_bytes(a[i].fmt, a[i].K),
                           mx_row_bytes(a[i].fmt, kQEl));
    j.dst[i] = make_stride(j.w[i], a[i].batch_stride * el, a[i].row_stride * el, kQEl * el);
  }
  if (!deal_blocks(j, n)) return cudaErrorInvalidValue;
#define STRATA_D(DT, FMT)                     \
  if (a->dst_dtype == DT && a->fmt == FMT)    \
    return n > 1 ? launch_blocks(mx_dequantize_kernel<DT, FMT, true>, j.first[3], st, j)    \
                 : launch_blocks(mx_dequantize_kernel<DT, FMT, false>, j.first[3], st, j);
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
  return launch_blocks(mx_tile_scales_kernel, (words + kQThreads - 1) / kQThreads, st, src, rows,
                       (int)(K / kMxBlock), (int)mx_ceil(K, 128), words,
                       reinterpret_cast<uint32_t*>(dst));
}

}  // namespace strata
