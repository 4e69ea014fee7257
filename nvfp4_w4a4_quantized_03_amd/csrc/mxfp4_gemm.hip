// Y = A B^T on MXFP4 operands for gfx950.
//
// The 4-bit matrix instructions take E2M1 operands with one E8M0 scale per 32
// elements of K, which is the format as it is stored: a lane's operand is 16
// bytes of codes (one block) of its row and the block's scale byte, and
// nothing is decoded.  Products and scales are exact; sums are binary32.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "internal.h"

namespace nvfp4 {
namespace {

constexpr int kOutF32 = 0;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ unsigned short bf16_bits(float f) {
  return __builtin_bit_cast(unsigned short, static_cast<__bf16>(f));
}

// Simple kernel for every shape: four waves of 32 x 32 outputs, operands from
// memory straight to registers, 64 of K an instruction.  Lane l has row l % 32
// and the block l / 32 of the two; a block past K is zeros.
template <int OUT>
__global__ void __launch_bounds__(256)
mxfp4_gemm_simple(const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales,
                  int64_t m, const uint8_t* __restrict__ b_codes,
                  const uint8_t* __restrict__ b_scales, int64_t n, int64_t k,
                  void* __restrict__ out, int64_t ldo, int64_t tiles_n) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m0 = blockIdx.x / tiles_n * 64 + (wave >> 1) * 32;
  const int64_t n0 = blockIdx.x % tiles_n * 64 + (wave & 1) * 32;
  const int r = lane & 31, h = lane >> 5;
  const int64_t blocks = k / 32;
  const int64_t ar = m0 + r < m ? m0 + r : m - 1, br = n0 + r < n ? n0 + r : n - 1;
  f32x16 acc = {};
  for (int64_t b0 = 0; b0 < blocks; b0 += 2) {
    const int64_t b = b0 + h;
    i32x8 av = {}, bv = {};
    unsigned as = 0, bs = 0;
    if (b < blocks) {
      const u32x4 a = *reinterpret_cast<const u32x4*>(a_codes + (ar * blocks + b) * 16);
      const u32x4 c = *reinterpret_cast<const u32x4*>(b_codes + (br * blocks + b) * 16);
      as = a_scales[ar * blocks + b];
      bs = b_scales[br * blocks + b];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        av[i] = static_cast<int>(a[i]);
        bv[i] = static_cast<int>(c[i]);
      }
    }
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc, 4, 4, 0, static_cast<int>(as),
                                                          0, static_cast<int>(bs));
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int64_t row = m0 + 8 * (e >> 2) + 4 * h + (e & 3), col = n0 + r;
    if (row < m && col < n) {
      if constexpr (OUT == kOutF32)
        static_cast<float*>(out)[row * ldo + col] = acc[e];
      else
        static_cast<unsigned short*>(out)[row * ldo + col] = bf16_bits(acc[e]);
    }
  }
}

}  // namespace

hipError_t launch_mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m,
                             const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k,
                             void* out, int out_dtype, int64_t ldo, hipStream_t stream) {
  const int64_t tm = (m + 63) / 64, tn = (n + 63) / 64;
  if (tm > 0xFFFFFF / tn) return hipErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(tm * tn);
  if (out_dtype == kOutF32)
    mxfp4_gemm_simple<0><<<grid, 256, 0, stream>>>(a_codes, a_scales, m, b_codes, b_scales, n, k,
                                                   out, ldo, tn);
  else
    mxfp4_gemm_simple<1><<<grid, 256, 0, stream>>>(a_codes, a_scales, m, b_codes, b_scales, n, k,
                                                   out, ldo, tn);
  return hipGetLastError();
}

}  // namespace nvfp4
