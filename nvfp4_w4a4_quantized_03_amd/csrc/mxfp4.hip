// MXFP4 tensors for gfx950: quantisation and the values of packed codes.
//
// Format (OCP microscaling, 4-bit form): E2M1 elements (1 sign, 2 exponent, 1
// mantissa bit: magnitudes 0 .5 1 1.5 2 3 4 6), one E8M0 scale 2^(byte - 127)
// per 32 consecutive elements of a row.  With m = max |x| of a block,
//   byte = max(floor(log2 m) - 2, -127) + 127 (0 for m = 0),
//   code = sign(x) | E2M1(|x| 2^(127 - byte)), nearest, ties to the even code,
//          saturating at 6.
// The scale is a power of two, so every step but the one rounding to E2M1 is
// exact in binary32: the exponent field of m is the logarithm, and the product
// with 2^(127 - byte) only moves it (below the normal range too: subnormals
// are kept, and where the product is lost the code is 0 either way).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kDtypeF32 = 0;
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// the largest of the quad of lanes that holds one block
__device__ __forceinline__ unsigned quad_max(unsigned x) {
  x = max(x, static_cast<unsigned>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0xB1, 0xF, 0xF, false)));
  return max(x, static_cast<unsigned>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x4E, 0xF, 0xF, false)));
}

// Scale byte of a block from the binary32 bits of its largest magnitude: the
// exponent field less 2, not below 0; 0xFF (NaN) if an infinity or NaN is
// among its values.
__device__ __forceinline__ unsigned scale_byte(unsigned bits) {
  const unsigned e = bits >> 23;
  return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// One piece of 8 elements a lane, a block a quad of lanes: a wave's loads and
// its code stores are contiguous.  Bound by memory: 32768 x 5120 bf16 (425 MB read
// and written) 74-78 us, 5.5-5.7 TB/s.
template <int DTYPE>
__global__ void __launch_bounds__(256)
mxfp4_quantize_kernel(const uint8_t* __restrict__ x, int64_t pieces, int64_t row_pieces,
                      int64_t ldx_bytes, uint8_t* __restrict__ codes,
                      uint8_t* __restrict__ scales) {
  constexpr int kPieceBytes = DTYPE == kDtypeF32 ? 32 : 16;
  const bool flat = ldx_bytes == row_pieces * kPieceBytes;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < pieces;
       t += stride) {
    const uint8_t* src = x + t * kPieceBytes;
    if (!flat) {
      const int64_t row = t / row_pieces;
      src = x + row * ldx_bytes + (t - row * row_pieces) * kPieceBytes;
    }
    float v[8];
    unsigned top = 0;
    if constexpr (DTYPE == kDtypeF32) {
      const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src));
      const u32x4 b = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src) + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[4 + i] = __uint_as_float(b[i]);
      }
    } else {
      const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(src));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    const unsigned byte = scale_byte(quad_max(top));
    const float r = __uint_as_float((254u - (byte < 254u ? byte : 253u)) << 23);
    unsigned c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * r, v[1] * r, 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * r, v[3] * r, 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * r, v[5] * r, 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * r, v[7] * r, 1.0f, 3);
    __builtin_nontemporal_store(c, reinterpret_cast<unsigned*>(codes) + t);
    if ((t & 3) == 0) scales[t >> 2] = static_cast<uint8_t>(byte);
  }
}

// binary32 value of a scale byte (0: 2^-127, subnormal; 255: NaN)
__device__ __forceinline__ float scale_value(unsigned byte) {
  return __uint_as_float(byte == 255u ? 0x7FC00000u : byte == 0u ? 0x00400000u : byte << 23);
}

// 16 bytes of output a lane (8 bf16 or 4 binary32 values).  e2m1 * 2^e has
// two significant bits: exact in both types, or past their range.  Bound by
// memory: 32768 x 5120 to bf16 72-77 us, 5.5-5.9 TB/s.
template <int DTYPE>
__global__ void __launch_bounds__(256)
mxfp4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                        int64_t pieces, int64_t row_pieces, void* __restrict__ out,
                        int64_t ldo_bytes) {
  constexpr int kShift = DTYPE == kDtypeF32 ? 3 : 2;     // pieces of a block: 8 or 4
  const bool flat = ldo_bytes == row_pieces * 16;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; t < pieces;
       t += stride) {
    const float s = scale_value(scales[t >> kShift]);
    uint8_t* dst = static_cast<uint8_t*>(out) + t * 16;
    if (!flat) {
      const int64_t row = t / row_pieces;
      dst = static_cast<uint8_t*>(out) + row * ldo_bytes + (t - row * row_pieces) * 16;
    }
    if constexpr (DTYPE == kDtypeF32) {
      const unsigned c = reinterpret_cast<const unsigned short*>(codes)[t];
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
      const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
      const f32x4 o = {a[0] * s, a[1] * s, b[0] * s, b[1] * s};
      __builtin_nontemporal_store(o, reinterpret_cast<f32x4*>(dst));
    } else {
      const unsigned c = reinterpret_cast<const unsigned*>(codes)[t];
      const f32x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3)};
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = (__float_as_uint(p[i][0] * s) >> 16) |
               (__float_as_uint(p[i][1] * s) & 0xFFFF0000u);
      __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(dst));
    }
  }
}

// a piece a lane; the loops in the kernels cover grids capped at the launch
// limit of 2^32 threads
unsigned grid_of(int64_t pieces) {
  const int64_t want = (pieces + 255) / 256;
  return static_cast<unsigned>(want < 0xFFFFFF ? want : 0xFFFFFF);
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, int x_dtype, int64_t rows, int64_t k, int64_t ldx,
                                 uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const int64_t row_pieces = k / 8, pieces = rows * row_pieces;
  const uint8_t* xb = static_cast<const uint8_t*>(x);
  if (x_dtype == kDtypeF32)
    mxfp4_quantize_kernel<0><<<grid_of(pieces), 256, 0, stream>>>(xb, pieces, row_pieces, ldx * 4,
                                                                  codes, scales);
  else
    mxfp4_quantize_kernel<1><<<grid_of(pieces), 256, 0, stream>>>(xb, pieces, row_pieces, ldx * 2,
                                                                  codes, scales);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                   int64_t k, void* out, int out_dtype, int64_t ldo,
                                   hipStream_t stream) {
  if (out_dtype == kDtypeF32) {
    const int64_t row_pieces = k / 4, pieces = rows * row_pieces;
    mxfp4_dequantize_kernel<0><<<grid_of(pieces), 256, 0, stream>>>(codes, scales, pieces,
                                                                    row_pieces, out, ldo * 4);
  } else {
    const int64_t row_pieces = k / 8, pieces = rows * row_pieces;
    mxfp4_dequantize_kernel<1><<<grid_of(pieces), 256, 0, stream>>>(codes, scales, pieces,
                                                                    row_pieces, out, ldo * 2);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
