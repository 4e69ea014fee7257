// Device helpers shared by the KV-cache kernels (fp8kv.hip, kvpage.hip,
// attention.hip): 16-element loads widened to binary32, the exact E4M3 cast
// of one 16-element group under a static decode scale, and division by a
// launch constant.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "formats.h"

namespace nvfp4 {
namespace {

constexpr int kDtypeF32 = 0;

// Quotients by a divisor that is fixed for a launch: floor(n / d) for
// 0 <= n < 2^31 as the high word of n * mul, shifted.  With l = floor(log2 d)
// and mul = ceil(2^(32 + l) / d) the error n (mul d - 2^(32 + l)) is below
// 2^31 d <= 2^(32 + l), so the quotient is exact.
struct FastDiv {
  unsigned d, mul, shift;
  static FastDiv of(unsigned d) {
    if (d == 1) return {1u, 0u, 0u};
    unsigned l = 0;
    while ((d >> l) > 1u) ++l;
    if ((d & (d - 1u)) == 0u) return {d, 0x80000000u, l - 1u};
    return {d, static_cast<unsigned>(((uint64_t(1) << (32 + l)) + d - 1) / d), l};
  }
  __device__ __forceinline__ unsigned div(unsigned n) const {
    return mul ? __umulhi(n, mul) >> shift : n;
  }
};

template <int DTYPE>
__device__ __forceinline__ void load16(const uint8_t* src, float* v) {
  if constexpr (DTYPE == kDtypeF32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 t = reinterpret_cast<const float4*>(src)[q];
      v[4 * q] = t.x; v[4 * q + 1] = t.y; v[4 * q + 2] = t.z; v[4 * q + 3] = t.w;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint4 t = reinterpret_cast<const uint4*>(src)[q];
      const unsigned w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * q + 2 * i] = __uint_as_float(w[i] << 16);
        v[8 * q + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
}

// Code magnitude of q = |x| / s with the bracketed hardware conversion of
// |x| r_lo and |x| r_hi (inputs clamped to 448, where the hardware would
// give NaN above 464); disagreement -> exact float64 settle.
__device__ __forceinline__ unsigned kv_code(float ax, float r_lo, float r_hi, double s) {
  const float lo = fminf(ax * r_lo, 448.0f), hi = fminf(ax * r_hi, 448.0f);
  const unsigned pk = static_cast<unsigned>(__builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, 0, false));
  const unsigned c = pk & 0xFFu;
  if (c == ((pk >> 8) & 0xFFu)) return c;
  return e4m3_settle(c, static_cast<double>(ax), s);
}

// Codes of one 16-element group, stored as one non-temporal 16-byte piece
// (the codes are a stream; a wave's stores cover 1 KiB).  `normal`: s within
// [2^-100, 2^100], where the bracketed conversion applies; otherwise every
// code is settled in float64 (or is 0 when s == 0).  Both flags are uniform,
// so the per-element work has no branch on them.
template <int DTYPE>
__device__ __forceinline__ void kv_cast_group(const uint8_t* src, uint8_t* dst, bool zero,
                                              bool normal, float r_lo, float r_hi,
                                              double sd) {
  float v[16];
  load16<DTYPE>(src, v);
  unsigned w[4] = {0u, 0u, 0u, 0u};
  if (normal) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const unsigned c = kv_code(__builtin_fabsf(v[i]), r_lo, r_hi, sd) |
                         ((__float_as_uint(v[i]) >> 24) & 0x80u);
      w[i >> 2] |= c << (8 * (i & 3));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const double ax = static_cast<double>(__builtin_fabsf(v[i]));
      const unsigned m = zero ? 0u : e4m3_settle(e4m3_candidate(ax / sd), ax, sd);
      const unsigned c = m | ((__float_as_uint(v[i]) >> 24) & 0x80u);
      w[i >> 2] |= c << (8 * (i & 3));
    }
  }
  typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 o = {w[0], w[1], w[2], w[3]};
  __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(dst));
}

}  // namespace
}  // namespace nvfp4
