// mx_abi.cu -- extern "C" entry points of the microscaled operators: argument
// checks and launches.  See include/strata_moe.h.
#include "abi_util.h"
#include "mx.cuh"
#include "qformat.cuh"

using namespace strata;

namespace {

bool valid_fmt(int32_t fmt) { return fmt == STRATA_MX_FP4 || fmt == STRATA_MX_FP8; }
bool valid_layout(int32_t l) { return l == STRATA_MX_ROWS || l == STRATA_MX_TILES; }

// What moe_mx_quantize and moe_mx_dequantize ask of a batch of matrices: the
// plain side (data, strides in elements) and the quantised one.
int32_t check_batch(const void* data, int32_t dtype, int64_t row_stride, int64_t batch_stride,
                    int32_t batch, int32_t rows, int32_t K, int32_t fmt, const void* codes,
                    uint64_t codes_stride, const void* scales, int32_t layout,
                    uint64_t scales_stride) {
  const int el = dtype_bytes(dtype);
  if (!el || !valid_fmt(fmt) || !valid_layout(layout)) return STRATA_EINVAL;
  if (batch < 0 || rows < 0 || K < kMxBlock || K % kMxBlock) return STRATA_EINVAL;
  if (row_stride < 0 || batch_stride < 0 || (rows > 1 && row_stride * el % 16) ||
      (batch > 1 && batch_stride * el % 16))
    return STRATA_EINVAL;
  const int64_t rows_p =
      layout == STRATA_MX_TILES ? mx_ceil(rows, kMxTileRows) * kMxTileRows : rows;
  if (batch * rows_p >= (int64_t)1 << 31) return STRATA_EINVAL;
  if (batch * rows_p * mx_ceil(K, 128) * 16 >= (int64_t)1 << 40) return STRATA_EINVAL;
  if (batch > 1 && (codes_stride < (uint64_t)(rows * mx_row_bytes(fmt, K)) || codes_stride % 16 ||
                    scales_stride < (uint64_t)mx_scale_plane(rows, K, layout) ||
                    (layout == STRATA_MX_TILES && scales_stride % 16)))
    return STRATA_EINVAL;
  if (batch == 0 || rows == 0) return STRATA_OK;
  if (!data || !codes || !scales || !aligned(data, 16) || !aligned(codes, 16) ||
      (layout == STRATA_MX_TILES && !aligned(scales, 16)))
    return STRATA_EINVAL;
  return STRATA_OK;
}

// The blobs of E MXFP4 experts.
int32_t check_experts(int32_t E, int32_t H, int32_t I, const void* blobs, uint64_t stride) {
  if (E < 0 || H < 128 || I < 128 || H % 128 || I % 128) return STRATA_EINVAL;
  uint64_t total = 0;
  plane_offsets(STRATA_FMT_MXFP4_32, H, I, &total);
  if (stride % 256 || stride < total) return STRATA_EINVAL;
  if (E > 0 && (!blobs || !aligned(blobs, 256))) return STRATA_EINVAL;
  return STRATA_OK;
}

}  // namespace

extern "C" {

uint64_t moe_mx_scale_bytes(int32_t rows, int32_t K, int32_t scale_layout) {
  if (rows < 0 || K < kMxBlock || K % kMxBlock || !valid_layout(scale_layout)) return 0;
  return (uint64_t)mx_scale_plane(rows, K, scale_layout);
}

int32_t moe_mx_quantize(const void* src, int32_t src_dtype, int32_t batch, int32_t rows, int32_t K,
                        int64_t src_row_stride, int64_t src_batch_stride, int32_t fmt, void* codes,
                        uint64_t codes_batch_stride, void* scales, int32_t scale_layout,
                        uint64_t scales_batch_stride, void* stream) {
  const int32_t r = check_batch(src, src_dtype, src_row_stride, src_batch_stride, batch, rows, K,
                                fmt, codes, codes_batch_stride, scales, scale_layout,
                                scales_batch_stride);
  if (r != STRATA_OK || batch == 0 || rows == 0) return r;
  MxQuantArgs a = {};
  a.src = src;
  a.src_dtype = src_dtype;
  a.batch = batch;
  a.rows = rows;
  a.K = K;
  a.row_stride = src_row_stride;
  a.batch_stride = src_batch_stride;
  a.fmt = fmt;
  a.codes = reinterpret_cast<uint8_t*>(codes);
  a.codes_stride = codes_batch_stride;
  a.scales = reinterpret_cast<uint8_t*>(scales);
  a.layout = scale_layout;
  a.scales_stride = scales_batch_stride;
  return from_cuda(launch_mx_quantize(&a, 1, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t moe_mx_dequantize(const void* codes, uint64_t codes_batch_stride, const void* scales,
                          int32_t scale_layout, uint64_t scales_batch_stride, int32_t fmt,
                          int32_t batch, int32_t rows, int32_t K, void* dst, int32_t dst_dtype,
                          int64_t dst_row_stride, int64_t dst_batch_stride, void* stream) {
  const int32_t r = check_batch(dst, dst_dtype, dst_row_stride, dst_batch_stride, batch, rows, K,
                                fmt, codes, codes_batch_stride, scales, scale_layout,
                                scales_batch_stride);
  if (r != STRATA_OK) return r;
  if ((rows > 1 && dst_row_stride < K) ||
      (batch > 1 && (dst_batch_stride < K ||
                     (dst_batch_stride < (rows - 1) * dst_row_stride + K &&
                      dst_row_stride < (batch - 1) * dst_batch_stride + K))))
    return STRATA_EINVAL;  // rows of dst would overlap
  if (batch == 0 || rows == 0) return STRATA_OK;
  MxDequantArgs a = {};
  a.codes = reinterpret_cast<const uint8_t*>(codes);
  a.codes_stride = codes_batch_stride;
  a.scales = reinterpret_cast<const uint8_t*>(scales);
  a.layout = scale_layout;
  a.scales_stride = scales_batch_stride;
  a.fmt = fmt;
  a.batch = batch;
  a.rows = rows;
  a.K = K;
  a.dst = dst;
  a.dst_dtype = dst_dtype;
  a.row_stride = dst_row_stride;
  a.batch_stride = dst_batch_stride;
  return from_cuda(launch_mx_dequantize(&a, 1, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t moe_mx_pack_experts(const void* gate, const void* up, const void* down, int32_t dtype,
                            const int64_t* row_strides, const int64_t* expert_strides, int32_t E,
                            int32_t H, int32_t I, void* blobs, uint64_t blob_stride,
                            void* stream) {
  const int32_t r = check_experts(E, H, I, blobs, blob_stride);
  if (r != STRATA_OK) return r;
  if (E == 0) return STRATA_OK;
  if (!row_strides || !expert_strides) return STRATA_EINVAL;
  const Planes pl = plane_offsets(STRATA_FMT_MXFP4_32, H, I);
  const void* src[3] = {gate, up, down};
  MxQuantArgs a[3] = {};
  for (int i = 0; i < 3; ++i) {
    a[i].src = src[i];
    a[i].src_dtype = dtype;
    a[i].batch = E;
    a[i].rows = i < 2 ? I : H;
    a[i].K = i < 2 ? H : I;
    a[i].row_stride = row_strides[i];
    a[i].batch_stride = expert_strides[i];
    a[i].fmt = STRATA_MX_FP4;
    a[i].codes = reinterpret_cast<uint8_t*>(blobs) + pl.codes[i];
    a[i].codes_stride = blob_stride;
    a[i].scales = reinterpret_cast<uint8_t*>(blobs) + pl.scales[i];
    a[i].layout = STRATA_MX_ROWS;
    a[i].scales_stride = blob_stride;
    const int32_t c = check_batch(src[i], dtype, a[i].row_stride, a[i].batch_stride, E,
                                  (int32_t)a[i].rows, (int32_t)a[i].K, a[i].fmt, a[i].codes,
                                  blob_stride, a[i].scales, a[i].layout, blob_stride);
    if (c != STRATA_OK) return c;
  }
  return from_cuda(launch_mx_quantize(a, 3, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t moe_mx_unpack_experts(const void* blobs, uint64_t blob_stride, int32_t E, int32_t H,
                              int32_t I, void* gate, void* up, void* down, int32_t dtype,
                              void* stream) {
  const int32_t r = check_experts(E, H, I, blobs, blob_stride);
  if (r != STRATA_OK) return r;
  if (E == 0) return STRATA_OK;
  const Planes pl = plane_offsets(STRATA_FMT_MXFP4_32, H, I);
  void* dst[3] = {gate, up, down};
  MxDequantArgs a[3] = {};
  for (int i = 0; i < 3; ++i) {
    a[i].codes = reinterpret_cast<const uint8_t*>(blobs) + pl.codes[i];
    a[i].codes_stride = blob_stride;
    a[i].scales = reinterpret_cast<const uint8_t*>(blobs) + pl.scales[i];
    a[i].layout = STRATA_MX_ROWS;
    a[i].scales_stride = blob_stride;
    a[i].fmt = STRATA_MX_FP4;
    a[i].batch = E;
    a[i].rows = i < 2 ? I : H;
    a[i].K = i < 2 ? H : I;
    a[i].dst = dst[i];
    a[i].dst_dtype = dtype;
    a[i].row_stride = a[i].K;
    a[i].batch_stride = (int64_t)H * I;
    const int32_t c = check_batch(dst[i], dtype, a[i].row_stride, a[i].batch_stride, E,
                                  (int32_t)a[i].rows, (int32_t)a[i].K, a[i].fmt, a[i].codes,
                                  blob_stride, a[i].scales, a[i].layout, blob_stride);
    if (c != STRATA_OK) return c;
  }
  return from_cuda(launch_mx_dequantize(a, 3, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t moe_mx_tile_scales(const void* scales, int32_t rows, int32_t K, void* tiles, void* stream) {
  if (rows < 0 || K < kMxBlock || K % kMxBlock) return STRATA_EINVAL;
  if (mx_scale_plane(rows, K, STRATA_MX_TILES) >= (int64_t)1 << 40) return STRATA_EINVAL;
  if (rows == 0) return STRATA_OK;
  if (!scales || !tiles || !aligned(tiles, 16)) return STRATA_EINVAL;
  return from_cuda(launch_mx_tile_scales(reinterpret_cast<const uint8_t*>(scales), rows, K,
                                         reinterpret_cast<uint8_t*>(tiles),
                                         reinterpret_cast<cudaStream_t>(stream)));
}

int32_t moe_add_rmsnorm(const void* x, int32_t x_dtype, const void* delta, int32_t delta_dtype,
                        const float* gain, int32_t T, int32_t H, float eps, void* residual_out,
                        void* out, int32_t out_dtype, int32_t mx_fmt, void* codes, void* scales,
                        int32_t scale_layout, void* stream) {
  if (T < 0 || H < 32 || H > 16384 || H % 8 || !(eps >= 0.f)) return STRATA_EINVAL;
  if (!dtype_bytes(x_dtype) || (delta && !dtype_bytes(delta_dtype)) ||
      (out && !dtype_bytes(out_dtype)))
    return STRATA_EINVAL;
  if (mx_fmt && (!valid_fmt(mx_fmt) || !valid_layout(scale_layout) || H % kMxBlock))
    return STRATA_EINVAL;
  if (T > (1 << 30)) return STRATA_EINVAL;
  if (T == 0) return STRATA_OK;
  if (!x || (!residual_out && !out && !mx_fmt) || (mx_fmt && (!codes || !scales)))
    return STRATA_EINVAL;
  if (!aligned(x, 16) || !aligned(delta, 16) || !aligned(gain, 16) || !aligned(residual_out, 16) ||
      !aligned(out, 16) || (mx_fmt && !aligned(codes, 16)) ||
      (mx_fmt && scale_layout == STRATA_MX_TILES && !aligned(scales, 16)))
    return STRATA_EINVAL;
  AddNormArgs a = {};
  a.x = x;
  a.x_dtype = x_dtype;
  a.delta = delta;
  a.delta_dtype = delta_dtype;
  a.gain = gain;
  a.T = T;
  a.H = H;
  a.eps = eps;
  a.inv_H = 1.0 / H;
  // squares lose at most 2^-150 each: 2^-55 of such a sum, 2^-50 of such an eps
  a.least = eps < 0x1p-100f ? (127u - 90u) << 23 : 0u;
  a.residual_out = residual_out;
  a.out = out;
  a.out_dtype = out_dtype;
  a.fmt = mx_fmt;
  a.codes = reinterpret_cast<uint8_t*>(codes);
  a.scales = reinterpret_cast<uint8_t*>(scales);
  a.layout = scale_layout;
  a.num_sms = num_sms_of_current_device();
  return from_cuda(launch_add_rmsnorm(a, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t moe_mx_linear(const void* x_codes, int32_t x_fmt, const void* x_scales, int32_t T,
                      const void* w_codes, int32_t w_fmt, const void* w_scales, int32_t N,
                      int32_t K, const float* bias, void* y, int32_t y_dtype, int64_t ldy,
                      int32_t* dev_status, void* stream) {
  const int el = dtype_bytes(y_dtype);
  if (!valid_fmt(x_fmt) || !valid_fmt(w_fmt) || !el) return STRATA_EINVAL;
  if (T < 0 || T > (1 << 22) || N < 1 || N > (1 << 24) || K < 128 || K > (1 << 24) || K % 128 ||
      ldy < N)
    return STRATA_EINVAL;
  if (x_fmt == STRATA_MX_FP4 && w_fmt == STRATA_MX_FP8) return STRATA_EUNSUPPORTED;
  if (T == 0) return STRATA_OK;
  if (!x_codes || !x_scales || !w_codes || !w_scales || !y) return STRATA_EINVAL;
  if (!aligned(x_codes, 32) || !aligned(w_codes, 32) || !aligned(x_scales, 16) ||
      !aligned(w_scales, 16) || !aligned(y, el) || !aligned(bias, 4))
    return STRATA_EINVAL;
  MxLinearArgs a = {};
  a.x_codes = reinterpret_cast<const uint8_t*>(x_codes);
  a.x_fmt = x_fmt;
  a.x_scales = reinterpret_cast<const uint8_t*>(x_scales);
  a.T = T;
  a.w_codes = reinterpret_cast<const uint8_t*>(w_codes);
  a.w_fmt = w_fmt;
  a.w_scales = reinterpret_cast<const uint8_t*>(w_scales);
  a.N = N;
  a.K = K;
  a.bias = bias;
  a.y = y;
  a.y_dtype = y_dtype;
  a.ldy = ldy;
  a.status = dev_status;
  a.num_sms = num_sms_of_current_device();
  const cudaError_t e = launch_mx_linear(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaErrorNotSupported ? STRATA_EUNSUPPORTED : from_cuda(e);
}

}  // extern "C"
