// add_rmsnorm.cu -- the residual's addition, root-mean-square norm and
// microscaled output in one pass:
//   r = x + delta;  h = r / sqrt(mean r^2 + eps) * gain;
//   residual_out = r;  out = round(h);  codes, scales = MX(h).
//
// One CTA a row, the row in registers between the sum of squares and the
// output, so every input is read once and every output written once: bound by
// HBM for many rows (T = 8192, H = 4096, fp32 + bf16 to bf16 and FP8: 66.9 us,
// 6.5 TB/s), by the launch and one load-reduce-store chain for few.  CTAs that
// take rows in turn, with the next rows copied ahead, are slower (98 us): a
// row's two reductions are the wait, and many CTAs hide it better than a few.
//
// A thread's up to 32 squares are summed in fp32, the threads' sums in fp64
// (fixed order: warp butterfly, warp partials), which leaves the mean to one
// rounding: a code next to a border between two then goes the way of the
// exact norm as often as 32 bits allow.
#include "mx.cuh"
#include "tc05.cuh"

namespace strata {

namespace {

constexpr int kNMaxThreads = 512;

// The row's groups of this thread, loaded before the first is used.
template <int DT, int VPT>
STRATA_DEVFN void load_groups(const void* p, int64_t base, int G, float (&v)[VPT][8]) {
  constexpr int kEl = DT == STRATA_DTYPE_F32 ? 4 : 2;
  const uint8_t* b = reinterpret_cast<const uint8_t*>(p) + base * kEl;
  Raw8<DT> raw[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int g = threadIdx.x + blockDim.x * j;
    if (g < G)
      raw[j].load(b + (int64_t)g * (8 * kEl));
    else
      raw[j].zero();
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) raw[j].values(v[j]);
}
STRATA_DEVFN void store8_as(void* p, int dt, int64_t i, const float (&v)[8]) {
  if (dt == STRATA_DTYPE_F32)
    store8<STRATA_DTYPE_F32>(reinterpret_cast<float*>(p) + i, v);
  else if (dt == STRATA_DTYPE_F16)
    store8<STRATA_DTYPE_F16>(reinterpret_cast<uint16_t*>(p) + i, v);
  else
    store8<STRATA_DTYPE_BF16>(reinterpret_cast<uint16_t*>(p) + i, v);
}

// VPT groups of 8 elements a thread: group threadIdx.x + blockDim.x * j.  XT,
// DT: dtypes of x and delta (DT < 0: no delta).
template <int XT, int DT, int VPT>
__global__ void __launch_bounds__(kNMaxThreads) add_rmsnorm_kernel(AddNormArgs a) {
  __shared__ double red[kNMaxThreads / 32];
  const int tid = threadIdx.x, nth = blockDim.x;
  const int G = a.H / 8;
  const int kt = (a.H + 127) / 128;
  const int row = blockIdx.x;
  pdl_wait_prior();
  if (row < a.T) {
    const int64_t base = (int64_t)row * a.H;
    float r[VPT][8];
    float ss = 0.f;
    load_groups<XT>(a.x, base, G, r);
    if constexpr (DT >= 0) {
      float d[VPT][8];
      load_groups<DT>(a.delta, base, G, d);
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) r[j][i] += d[j][i];
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int g = tid + nth * j;
      if (a.residual_out && g < G)
        store8<XT>(reinterpret_cast<uint8_t*>(a.residual_out) +
                       (base + 8 * g) * (XT == STRATA_DTYPE_F32 ? 4 : 2),
                   r[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(r[j][i], r[j][i], ss);
    }
    double sum = ss;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    sum = (tid & 31) < nth / 32 ? red[tid & 31] : 0.;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sum = __shfl_sync(0xffffffffu, sum, 0);
    const float inv = rsqrtf((float)sum * (1.0f / (float)a.H) + a.eps);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int g = tid + nth * j;
      float h[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = r[j][i] * inv;
      if (a.gain && g < G) {
        float w[8];
        load8<STRATA_DTYPE_F32>(a.gain + 8 * g, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] *= w[i];
      }
      if (a.out && g < G) store8_as(a.out, a.out_dtype, base + 8 * g, h);
      if (a.fmt) {
        // four adjacent lanes hold a block of 32
        uint32_t m = max_bits8(h);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        uint2 c;
        uint32_t e;
        if (a.fmt == STRATA_MX_FP4) {
          e = mx_scale_of<STRATA_MX_FP4>(m);
          c = mx_encode8<STRATA_MX_FP4>(h, e);
        } else {
          e = mx_scale_of<STRATA_MX_FP8>(m);
          c = mx_encode8<STRATA_MX_FP8>(h, e);
        }
        if (g < G) {
          if (a.fmt == STRATA_MX_FP4)
            reinterpret_cast<uint32_t*>(a.codes)[base / 8 + g] = c.x;
          else
            reinterpret_cast<uint2*>(a.codes)[base / 8 + g] = c;
          if ((tid & 3) == 0) {
            if (a.layout == STRATA_MX_TILES)
              a.scales[mx_tile_byte(row, g / 4, kt)] = (uint8_t)e;
            else
              a.scales[(base + 8 * g) / kMxBlock] = (uint8_t)e;
          }
        }
      }
    }
  }
  // padding of the scale tiles: the last blocks of every row, and the rows
  // behind the last
  if (a.fmt && a.layout == STRATA_MX_TILES) {
    for (int b = (row < a.T ? a.H / kMxBlock : 0) + tid; b < kt * kMxTileBlocks; b += nth)
      a.scales[mx_tile_byte(row, b, kt)] = 0;
  }
}

template <int XT, int DT, int VPT>
cudaError_t launch_norm(const AddNormArgs& a, int rows, int threads, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(rows);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, add_rmsnorm_kernel<XT, DT, VPT>, a);
}

template <int XT, int VPT>
cudaError_t launch_norm_d(const AddNormArgs& a, int rows, int threads, cudaStream_t st) {
  if (!a.delta) return launch_norm<XT, -1, VPT>(a, rows, threads, st);
  if (a.delta_dtype == STRATA_DTYPE_F32)
    return launch_norm<XT, STRATA_DTYPE_F32, VPT>(a, rows, threads, st);
  if (a.delta_dtype == STRATA_DTYPE_F16)
    return launch_norm<XT, STRATA_DTYPE_F16, VPT>(a, rows, threads, st);
  return launch_norm<XT, STRATA_DTYPE_BF16, VPT>(a, rows, threads, st);
}
template <int VPT>
cudaError_t launch_norm_x(const AddNormArgs& a, int rows, int threads, cudaStream_t st) {
  if (a.x_dtype == STRATA_DTYPE_F32)
    return launch_norm_d<STRATA_DTYPE_F32, VPT>(a, rows, threads, st);
  if (a.x_dtype == STRATA_DTYPE_F16)
    return launch_norm_d<STRATA_DTYPE_F16, VPT>(a, rows, threads, st);
  return launch_norm_d<STRATA_DTYPE_BF16, VPT>(a, rows, threads, st);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormArgs& a, cudaStream_t st) {
  const int rows = a.fmt && a.layout == STRATA_MX_TILES
                       ? (int)(mx_ceil(a.T, kMxTileRows) * kMxTileRows)
                       : a.T;
  // One group a thread, or two (32 bytes of a 16-bit x) where there are rows
  // enough to fill the SMs: T = 4096, H = 4096, bf16 to FP4 24.4 us with one,
  // 21.5 with two; T = 16: 2.5 and 2.8; fp32 rows 66.9 and 67.8 (T = 8192).
  const int G = a.H / 8;
  int vpt = a.x_dtype != STRATA_DTYPE_F32 && a.T > 148 ? 2 : 1;
  while (G > vpt * kNMaxThreads) vpt *= 2;
  const int threads = (((G + vpt - 1) / vpt) + 31) & ~31;
  if (vpt == 1) return launch_norm_x<1>(a, rows, threads, st);
  if (vpt == 2) return launch_norm_x<2>(a, rows, threads, st);
  return launch_norm_x<4>(a, rows, threads, st);
}

}  // namespace strata
