// add_rmsnorm.cu -- the residual's addition, root-mean-square norm and
// microscaled output in one pass:
//   r = x + delta;  h = r / sqrt(mean r^2 + eps) * gain;
//   residual_out = r;  out = round(h);  codes, scales = MX(h).
//
// A row is one CTA's, or one or two warps' of a CTA of 128 threads, and stays
// in registers between the sum of squares and the output, so every input is
// read once and every output written once: bound by HBM for many rows (T =
// 8192, H = 4096, fp32 + bf16 to bf16 and FP8: 66.0 us, 6.6 TB/s), by
// instructions where a row is only read and its codes written (126 a group of
// 8 elements and warp; T = 5859, H = 4096, bf16 to FP4: 18.6 us), by the
// launch and one load-reduce-store chain for few.  CTAs that take rows in
// turn, with the next rows copied ahead, are slower (98 us for 66.0): a row's
// two reductions are the wait, and many CTAs hide it better than a few.
//
// A thread's up to 32 squares are summed in fp32, in two sums, the threads' sums
// in fp64 (fixed order: warp butterfly, warp partials), and the mean with eps is
// rounded to fp32 once: a code next to a border between two then goes the way
// of the exact norm as often as 32 bits allow.  A thread whose squares leave
// fp32's range, or, where eps is too small to cover it, are so small that they
// lose bits, squares r times a power of two; a row whose mean is out there is
// taken nearer to one in the same way.  The two checks and the mean in fp64 cost
// 0 to 3 % (T = 93750, H = 256 21.4 us for 20.7, T = 8192 nothing) and 0.1 us of
// a few rows' 2.0; summing such rows' threads a second time instead takes
// barriers by number, of which an SM has few (40 us for T = 93750).
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

// Whether a sum of squares is one from `least` (its bits) to 2^127: bits order
// like the numbers, NaN's are above all.
STRATA_DEVFN bool within(float sum, uint32_t least) {
  return __float_as_uint(sum) - least <= __float_as_uint(0x1p127f) - least;
}
// What brings values whose squares leave fp32's range back into it: below,
// those of a sum under 2^-90 (r < 2^-43 where a mean is under 2^-100, H <=
// 2^14) stay under 2^57; above, all stay under 2^58, and what an element loses
// is below 2^-120 of the row's root mean square.
STRATA_DEVFN float nearer_to_one(float square) { return square < 1.f ? 0x1p100f : 0x1p-70f; }

// A group of 8 as codes, and its block's scale byte (four adjacent lanes hold
// a block).
template <int FMT>
STRATA_DEVFN void put_mx(const AddNormArgs& a, const float (&h)[8], int64_t group, uint8_t* scale,
                         bool some) {
  uint32_t m = max_bits8(h);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t e = mx_scale_of<FMT>(m);
  const uint2 c = mx_encode8<FMT>(h, e);
  if (!some) return;
  if constexpr (FMT == STRATA_MX_FP4)
    reinterpret_cast<uint32_t*>(a.codes)[group] = c.x;
  else
    reinterpret_cast<uint2*>(a.codes)[group] = c;
  if (threadIdx.x % 4 == 0) *scale = (uint8_t)e;
}

// A row is blockDim.x threads', VPT groups of 8 elements each: group threadIdx.x
// + blockDim.x * j; a CTA has blockDim.y rows.  XT, DT: dtypes of x and delta
// (DT < 0: no delta).
template <int XT, int DT, int VPT>
__global__ void __launch_bounds__(kNMaxThreads) add_rmsnorm_kernel(AddNormArgs a) {
  __shared__ double red[kNMaxThreads / 32];
  const int tid = threadIdx.x, nth = blockDim.x;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  const int G = row < a.T ? a.H / 8 : 0;
  pdl_wait_prior();
  const int64_t base = (int64_t)row * a.H;
  float r[VPT][8];
  float even = 0.f, odd = 0.f;  // sums of squares
  load_groups<XT>(a.x, base, G, r);
  if constexpr (DT >= 0) {
    float d[VPT][8];
    load_groups<DT>(a.delta, base, G, d);
#pragma unroll
    for (int j = 0; j < VPT; ++j) add8(r[j], d[j]);
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int g = tid + nth * j;
    if (a.residual_out && g < G)
      store8<XT>(reinterpret_cast<uint8_t*>(a.residual_out) +
                     (base + 8 * g) * (XT == STRATA_DTYPE_F32 ? 4 : 2),
                 r[j]);
    squares8(r[j], even, odd);
  }
  double sum = (double)even + odd;
  if (__any_sync(0xffffffffu, !within(even + odd, a.least))) {
    const float s = within(even + odd, a.least) ? 1.f : nearer_to_one(even + odd);
    even = odd = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float q[8];
      scale8(r[j], s, q);
      squares8(q, even, odd);
    }
    sum = ((double)even + odd) * (s < 1.f ? 0x1p140 : s > 1.f ? 0x1p-200 : 1.);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (nth > 32) {
    double* part = red + threadIdx.y * (nth / 32);
    if ((tid & 31) == 0) part[tid >> 5] = sum;
    __syncthreads();
    sum = (tid & 31) < nth / 32 ? part[tid & 31] : 0.;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    sum = __shfl_sync(0xffffffffu, sum, 0);
  }
  const int kt = (a.H + 127) / 128;
  const bool tiles = a.fmt && a.layout == STRATA_MX_TILES;
  uint8_t* const scales = a.scales + (tiles ? mx_tile_row(row, kt) : base / kMxBlock);
  sum = sum * a.inv_H + a.eps;
  float mean = (float)sum;
  if (!within(mean, __float_as_uint(0x1p-100f))) {
    const float s = nearer_to_one(mean);  // h is also that of r s and eps s^2
    mean = (float)(sum * s * s);
#pragma unroll
    for (int j = 0; j < VPT; ++j) scale8(r[j], s, r[j]);
  }
  const float inv = rsqrtf(mean);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int g = tid + nth * j;
    float h[8];
    scale8(r[j], inv, h);
    if (a.gain && g < G) {
      float w[8];
      load8<STRATA_DTYPE_F32>(a.gain + 8 * g, w);
      mul8(h, w, h);
    }
    if (a.out && g < G) store8_as(a.out, a.out_dtype, base + 8 * g, h);
    uint8_t* const scale = scales + (tiles ? mx_tile_block(g / 4) : g / 4);
    if (a.fmt == STRATA_MX_FP4)
      put_mx<STRATA_MX_FP4>(a, h, base / 8 + g, scale, g < G);
    else if (a.fmt == STRATA_MX_FP8)
      put_mx<STRATA_MX_FP8>(a, h, base / 8 + g, scale, g < G);
  }
  // padding of the scale tiles: the last blocks of every row, and the rows
  // behind the last (the grid ends with the last tile's)
  if (tiles)
    for (int b = G / 4 + tid; b < kt * kMxTileBlocks; b += nth) scales[mx_tile_block(b)] = 0;
}

template <int XT, int DT, int VPT>
cudaError_t launch_norm(const AddNormArgs& a, int rows, dim3 block, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((rows + block.y - 1) / block.y);
  cfg.blockDim = block;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, add_rmsnorm_kernel<XT, DT, VPT>, a);
}

template <int XT, int VPT>
cudaError_t launch_norm_d(const AddNormArgs& a, int rows, dim3 block, cudaStream_t st) {
  if (!a.delta) return launch_norm<XT, -1, VPT>(a, rows, block, st);
  if (a.delta_dtype == STRATA_DTYPE_F32)
    return launch_norm<XT, STRATA_DTYPE_F32, VPT>(a, rows, block, st);
  if (a.delta_dtype == STRATA_DTYPE_F16)
    return launch_norm<XT, STRATA_DTYPE_F16, VPT>(a, rows, block, st);
  return launch_norm<XT, STRATA_DTYPE_BF16, VPT>(a, rows, block, st);
}
template <int VPT>
cudaError_t launch_norm_x(const AddNormArgs& a, int rows, dim3 block, cudaStream_t st) {
  if (a.x_dtype == STRATA_DTYPE_F32)
    return launch_norm_d<STRATA_DTYPE_F32, VPT>(a, rows, block, st);
  if (a.x_dtype == STRATA_DTYPE_F16)
    return launch_norm_d<STRATA_DTYPE_F16, VPT>(a, rows, block, st);
  return launch_norm_d<STRATA_DTYPE_BF16, VPT>(a, rows, block, st);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const AddNormArgs& a, cudaStream_t st) {
  const int rows = a.fmt && a.layout == STRATA_MX_TILES
                       ? (int)(mx_ceil(a.T, kMxTileRows) * kMxTileRows)
                       : a.T;
  const int G = a.H / 8;
  const int64_t groups = (int64_t)a.T * G;
  // Groups a thread: one where that leaves SMs half empty (a thread's chain is
  // the time: T = 234, H = 1024, bf16 to FP4 2.0 us, with two 2.3) and for
  // rows of one warp; else two, which share a thread's fixed part (T = 2343:
  // 4.0 and 3.6 us).  With the SMs filled several times over, rows that are
  // only read are bound by instructions, four save more of them (T = 23437:
  // 23.5, 19.0 and 17.0 us with one, two and four), and fp32 rows with a
  // delta by HBM (T = 5859, H = 4096: 48.1, 49.0 and 50.7 us).
  const int64_t filled = (int64_t)a.num_sms * 64 * 32;
  int vpt = 1;
  if (G > 32 && groups > filled / 2) vpt = 2;
  if (vpt == 2 && groups > 4 * filled)
    vpt = !a.delta ? (G > 64 ? 4 : 2) : a.x_dtype == STRATA_DTYPE_F32 ? 1 : 2;
  // threads of a row, whole warps; not an eighth more idle ones than with half
  // of the groups (T = 15625, H = 1536, four groups: 21.5 us, two: 19.1 us)
  auto threads_of = [&](int v) { return ((G + v - 1) / v + 31) & ~31; };
  while (vpt > 1 && 8 * vpt * threads_of(vpt) > 9 * (vpt / 2) * threads_of(vpt / 2)) vpt /= 2;
  while (G > vpt * kNMaxThreads) vpt *= 2;
  const int threads = threads_of(vpt);
  // up to 128 threads a CTA, then a CTA a row (T = 93750, H = 256, bf16 to
  // FP4: 21 us with four rows a CTA, 50 with one)
  int per = 1;
  while (2 * per * threads <= 128) per *= 2;
  const dim3 block(threads, per);
  if (vpt == 1) return launch_norm_x<1>(a, rows, block, st);
  if (vpt == 2) return launch_norm_x<2>(a, rows, block, st);
  return launch_norm_x<4>(a, rows, block, st);
}

}  // namespace strata
