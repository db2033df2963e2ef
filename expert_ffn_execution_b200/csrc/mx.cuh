// mx.cuh -- microscaled (OCP MX v1.0) rows: blocks of 32 consecutive elements
// with one E8M0 scale byte, elements E2M1 (two a byte, low nibble first) or
// E4M3, and the internal interfaces of the calls that make and read them.
#pragma once

#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace strata {

constexpr int kMxBlock = 32;
// A scale tile: 128 rows x 4 blocks (128 elements of K), 512 bytes, in the
// order in which the tensor core wants the scales in tensor memory: 32 lanes
// of 16 bytes, lane = row % 32, then row / 32, then the block.
constexpr int kMxTileRows = 128;
constexpr int kMxTileBlocks = 4;
constexpr int kMxTileBytes = kMxTileRows * kMxTileBlocks;

__host__ __device__ inline int64_t mx_row_bytes(int fmt, int64_t K) {
  return fmt == STRATA_MX_FP4 ? K / 2 : K;
}
__host__ __device__ inline int64_t mx_ceil(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ inline int64_t mx_scale_plane(int64_t rows, int64_t K, int layout) {
  return layout == STRATA_MX_TILES
             ? mx_ceil(rows, kMxTileRows) * mx_ceil(K, kMxTileBlocks * kMxBlock) * kMxTileBytes
             : rows * (K / kMxBlock);
}
// Byte of (row, block) in a plane of `kt` scale tiles a row of tiles: the
// row's part and the block's.
__host__ __device__ inline int64_t mx_tile_row(uint32_t row, uint32_t kt) {
  return (int64_t)((uint64_t)(row / kMxTileRows) * kt * kMxTileBytes) +
         (row % 32 * 16 + row / 32 % 4 * 4);
}
__host__ __device__ inline int64_t mx_tile_block(uint32_t block) {
  return (int64_t)(block / kMxTileBlocks) * kMxTileBytes + block % kMxTileBlocks;
}
__host__ __device__ inline int64_t mx_tile_byte(uint32_t row, uint32_t block, uint32_t kt) {
  return mx_tile_row(row, kt) + mx_tile_block(block);
}

// ---------------------------------------------------------------- 8 elements
// Eight consecutive elements of a tensor of dtype DT (16-byte aligned), as
// loaded.
template <int DT>
struct Raw8 {
  uint4 w[DT == STRATA_DTYPE_F32 ? 2 : 1];
  STRATA_DEVFN void zero() {
    for (uint4& q : w) q = make_uint4(0u, 0u, 0u, 0u);
  }
  STRATA_DEVFN void load(const void* p) {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(w) / 16); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  STRATA_DEVFN void values(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(w) / 16); ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (DT == STRATA_DTYPE_F32) {
          v[4 * i + j] = __uint_as_float(u[j]);
        } else if constexpr (DT == STRATA_DTYPE_BF16) {
          v[2 * j] = __uint_as_float(u[j] << 16);
          v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        } else {
          const float2 f = __half22float2(u32_as_h2(u[j]));
          v[2 * j] = f.x;
          v[2 * j + 1] = f.y;
        }
      }
    }
  }
  // The largest magnitude as fp32 bits (16-bit types: two at a time as they
  // are stored, whose bits order like the magnitudes too).
  STRATA_DEVFN uint32_t max_bits(const float (&v)[8]) const;
};
template <int DT>
STRATA_DEVFN void load8(const void* p, float (&v)[8]) {
  Raw8<DT> r;
  r.load(p);
  r.values(v);
}

// Eight products, two an instruction; c may be a.
STRATA_DEVFN void mul8(const float (&a)[8], const float (&b)[8], float (&c)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "=f"(c[i]), "=f"(c[i + 1])
        : "f"(a[i]), "f"(a[i + 1]), "f"(b[i]), "f"(b[i + 1]));
}
STRATA_DEVFN void scale8(const float (&a)[8], float s, float (&c)[8]) {
  const float b[8] = {s, s, s, s, s, s, s, s};
  mul8(a, b, c);
}
// a += b, and two running sums of squares.
STRATA_DEVFN void add8(float (&a)[8], const float (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a[i]), "+f"(a[i + 1])
        : "f"(b[i]), "f"(b[i + 1]));
}
STRATA_DEVFN void squares8(const float (&a)[8], float& even, float& odd) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("{\n\t.reg .b64 a, s;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 s, {%0, %1};\n\t"
        "fma.rn.f32x2 s, a, a, s;\n\tmov.b64 {%0, %1}, s;\n\t}"
        : "+f"(even), "+f"(odd)
        : "f"(a[i]), "f"(a[i + 1]));
}

// Two values rounded to nearest even in the 16-bit type DT, first one low.
template <int DT>
STRATA_DEVFN uint32_t pack2(float a, float b) {
  if constexpr (DT == STRATA_DTYPE_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return h2_as_u32(__floats2half2_rn(a, b));
  }
}

template <int DT>
STRATA_DEVFN void store8(void* p, const float (&v)[8]) {
  if constexpr (DT == STRATA_DTYPE_F32) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]),
                   pack2<DT>(v[6], v[7]));
  }
}

// ---------------------------------------------------------------- one block
// The scale byte of a block from the largest of its magnitudes as fp32 bits,
// which order like the magnitudes, Inf and NaN above every number.
// floor(log2 m) is their exponent field, so e = field - emax, at least 0;
// subnormal m has field 0 and lands on e = 0 as the clamp asks.  A block with
// Inf or NaN is NaN.
template <int FMT>
STRATA_DEVFN uint32_t mx_scale_of(uint32_t m) {
  constexpr int kEmax = FMT == STRATA_MX_FP4 ? 2 : 8;
  return m >= 0x7f800000u ? 255u : (uint32_t)max((int)(m >> 23) - kEmax, 0);
}
// Eight codes under scale byte e: FP4 in .x, FP8 in .x and .y.  x * 2^(127-e)
// is exact but for results below the smallest element, which round to zero
// either way.
template <int FMT>
STRATA_DEVFN uint2 mx_encode8(const float (&v)[8], uint32_t e) {
  uint2 codes = make_uint2(0u, 0u);
  const float s = __uint_as_float((254u - e) << 23);  // not used for e = 255
  float x[8];
  scale8(v, s, x);
  // the conversions' pairs are joined as registers of 8 and 16 bits (joined by
  // shifts, 52M bf16 to MXFP4 took 24.2 us for 22.6)
  if constexpr (FMT == STRATA_MX_FP4) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(codes.x)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]),
          "f"(x[5]), "f"(x[6]), "f"(x[7]));
  } else {
    asm("{\n\t.reg .b16 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %3, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 b, %5, %4;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 c, %7, %6;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 d, %9, %8;\n\t"
        "mov.b32 %0, {a, b};\n\t"
        "mov.b32 %1, {c, d};\n\t}"
        : "=r"(codes.x), "=r"(codes.y)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]),
          "f"(x[5]), "f"(x[6]), "f"(x[7]));
  }
  return e == 255u ? make_uint2(0u, 0u) : codes;
}
STRATA_DEVFN float max3(float a, float b, float c) {  // NaN where one is
  float m;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
// Bits of the largest magnitude; above every number's where one is NaN.
STRATA_DEVFN uint32_t max_bits8(const float (&v)[8]) {
  const float m = max3(fabsf(v[0]), fabsf(v[1]), fabsf(v[2]));
  const float n = max3(fabsf(v[3]), fabsf(v[4]), fabsf(v[5]));
  return __float_as_uint(max3(max3(m, n, fabsf(v[6])), fabsf(v[7]), 0.f));
}

template <int DT>
STRATA_DEVFN uint32_t Raw8<DT>::max_bits(const float (&v)[8]) const {
  if constexpr (DT == STRATA_DTYPE_F32) {
    return max_bits8(v);
  } else {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    const uint32_t m = __vimax3_u16x2(
        __vimax3_u16x2(w[0].x & kAbs, w[0].y & kAbs, w[0].z & kAbs), w[0].w & kAbs, 0u);
    const uint32_t h = max(m & 0xffffu, m >> 16);
    if constexpr (DT == STRATA_DTYPE_BF16)
      return h << 16;
    else
      return __float_as_uint(__half2float(__ushort_as_half((uint16_t)h))) & 0x7fffffffu;
  }
}

// 2^(e-127) in fp32 (2^-127 is a subnormal; 255 is NaN).
STRATA_DEVFN float mx_scale_value(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7fc00000u : e == 0u ? 0x00400000u : e << 23);
}

// Eight codes -> values; exact in fp32 down to 2^-136, the smallest E4M3
// step under the smallest scale.
template <int FMT>
STRATA_DEVFN void mx_decode8(uint2 codes, uint32_t e, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2_raw h;
    if constexpr (FMT == STRATA_MX_FP4) {
      h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)(codes.x >> (8 * i)), __NV_E2M1);
    } else {
      const uint32_t w = i < 2 ? codes.x : codes.y;
      h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (i & 1))), __NV_E4M3);
    }
    const float2 f = __half22float2(__half2(h));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
  scale8(v, mx_scale_value(e), v);
}

// ---------------------------------------------------------------- interfaces
struct MxQuantArgs {
  const void* src;
  int src_dtype;
  int64_t batch, rows, K;
  int64_t row_stride, batch_stride;  // elements
  int fmt;
  uint8_t* codes;
  uint64_t codes_stride;  // bytes between matrices
  uint8_t* scales;
  int layout;
  uint64_t scales_stride;  // bytes between matrices
};
// n <= 3 batches of one dtype and format in one launch.
cudaError_t launch_mx_quantize(const MxQuantArgs* a, int n, cudaStream_t st);

struct MxDequantArgs {
  const uint8_t* codes;
  uint64_t codes_stride;
  const uint8_t* scales;
  int layout;
  uint64_t scales_stride;
  int fmt;
  int64_t batch, rows, K;
  void* dst;
  int dst_dtype;
  int64_t row_stride, batch_stride;  // elements
};
cudaError_t launch_mx_dequantize(const MxDequantArgs* a, int n, cudaStream_t st);
cudaError_t launch_mx_tile_scales(const uint8_t* src, int64_t rows, int64_t K, uint8_t* dst,
                                  cudaStream_t st);

struct AddNormArgs {
  const void* x;
  int x_dtype;
  const void* delta;  // or nullptr
  int delta_dtype;
  const float* gain;  // or nullptr
  int T, H;
  double eps, inv_H;
  uint32_t least;      // bits of the least sum of squares of a thread that loses none
  void* residual_out;  // dtype of x, or nullptr
  void* out;           // or nullptr
  int out_dtype;
  int fmt;  // 0: no codes
  uint8_t* codes;
  uint8_t* scales;
  int layout;
  int num_sms;
};
cudaError_t launch_add_rmsnorm(const AddNormArgs& a, cudaStream_t st);

struct MxLinearArgs {
  const uint8_t* x_codes;
  int x_fmt;
  const uint8_t* x_scales;
  int T;
  const uint8_t* w_codes;
  int w_fmt;
  const uint8_t* w_scales;
  int N, K;
  const float* bias;  // or nullptr
  void* y;
  int y_dtype;
  int64_t ldy;
  int32_t* status;
  int num_sms;
};
cudaError_t launch_mx_linear(const MxLinearArgs& a, cudaStream_t st);
cudaError_t launch_mx_gemm(const MxLinearArgs& a, cudaStream_t st);

}  // namespace strata
