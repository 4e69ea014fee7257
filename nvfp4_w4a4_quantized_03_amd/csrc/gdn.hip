// Linear attention with a decay for each head, with or without the delta rule
// (the recurrence of a Gated DeltaNet layer), for gfx950.
//
// For each request and value head, over its tokens in order, with the state S
// [dk][dv] in binary32:
//   S <- alpha S,  u = beta (v - S^T k)  (plain rule: u = v),
//   S <- S + k u^T,  o = scale S^T q.
//
// One pass over S a token: with a = S^T k and b = S^T q of the old state,
//   u = beta (v - alpha a),  o = scale (alpha b + (k.q) u).
// A column of S depends on no other column, so a wave owns 16 columns and all
// rows, and nothing is exchanged between waves.  The state passes once in and
// once out, whatever the tokens in between; for single tokens that is all there
// is to move, and the kernel is bound by it.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "internal.h"

namespace nvfp4 {
namespace {

typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr float kNormEps = 1e-6f;

struct GdnArgs {
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;   // bytes
  const float* alpha;
  const float* beta;                  // nullptr: the plain rule
  int64_t ld_alpha, ld_beta;
  uint8_t* out;
  int64_t out_token, out_head;        // bytes
  float* state;
  int64_t n_slots, slot_stride;
  const int32_t* slots;
  const int32_t* cu;
  const int32_t* cached;
  int n_tokens, n_requests, n_heads, group, dv;
  float scale;
  int normalize;
};

__device__ __forceinline__ float bf16_value(unsigned short x) {
  return __uint_as_float(static_cast<unsigned>(x) << 16);
}

__device__ __forceinline__ unsigned short bf16_bits(float f) {
  return __builtin_bit_cast(unsigned short, static_cast<__bf16>(f));
}

// Sum over the 16 lanes that share lane & 3; every one of them gets it.
__device__ __forceinline__ float sum_rows(float x) {
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x124, 0xF, 0xF, false));
  x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x128, 0xF, 0xF, false));
  unsigned u = __float_as_uint(x);
  auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  u = __float_as_uint(x);
  r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The rows of request r, or an empty range if it has none or is left out; a
// slot out of range leaves it out.
struct Request {
  int first, len;
  int64_t slot;
  bool fresh;
};
__device__ __forceinline__ Request request_of(const GdnArgs& a, int r) {
  const int lo = max(a.cu[r], 0), hi = min(a.cu[r + 1], a.n_tokens);
  const int64_t slot = a.slots ? a.slots[r] : r;
  const bool held = slot >= 0 && slot < a.n_slots;
  return {lo, held && hi > lo ? hi - lo : 0, held ? slot : 0, a.cached && a.cached[r] <= 0};
}

// Token after token.  Lane l has the dk / 16 rows from dk / 16 * (l / 4) and
// the four columns from 4 (l % 4) of its wave's 16.
template <int DK, bool DELTA>
__global__ void __launch_bounds__(256)
gdn_tokens_kernel(const GdnArgs a) {
  constexpr int R = DK / 16;
  const int lane = threadIdx.x & 63;
  const int slices = (a.dv + 63) >> 6;
  const int c0 = (blockIdx.x % slices * 4 + (threadIdx.x >> 6)) * 16;
  if (c0 >= a.dv) return;
  const int rh = blockIdx.x / slices;
  const int r = rh / a.n_heads, h = rh - r * a.n_heads, hk = h / a.group;
  const Request rq = request_of(a, r);
  if (rq.len == 0) return;
  const int row0 = (lane >> 2) * R, col = c0 + (lane & 3) * 4;
  float* sp = a.state + rq.slot * a.slot_stride + (static_cast<int64_t>(h) * DK + row0) * a.dv + col;
  f32x4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    s[i] = rq.fresh ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : *reinterpret_cast<const f32x4*>(sp + i * a.dv);
  for (int t = rq.first; t < rq.first + rq.len; ++t) {
    typedef unsigned short row_t __attribute__((ext_vector_type(R)));
    const row_t kr = *reinterpret_cast<const row_t*>(a.k + t * a.k_token + hk * a.k_head + row0 * 2);
    const row_t qr = *reinterpret_cast<const row_t*>(a.q + t * a.q_token + hk * a.q_head + row0 * 2);
    const u16x4 vr = *reinterpret_cast<const u16x4*>(a.v + t * a.v_token + h * a.v_head + col * 2);
    const float al = a.alpha[t * a.ld_alpha + h];
    float kv[R], qv[R];
    f32x4 ks = {}, qs = {};
    float kq = 0.0f, kk = 0.0f, qq = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      kv[i] = bf16_value(kr[i]);
      qv[i] = bf16_value(qr[i]);
      kq = __builtin_fmaf(kv[i], qv[i], kq);
      kk = __builtin_fmaf(kv[i], kv[i], kk);
      qq = __builtin_fmaf(qv[i], qv[i], qq);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (DELTA) ks[j] = __builtin_fmaf(kv[i], s[i][j], ks[j]);
        qs[j] = __builtin_fmaf(qv[i], s[i][j], qs[j]);
      }
    }
    kq = sum_rows(kq);
    float rk = 1.0f, rqn = a.scale;
    if (a.normalize) {
      rk = 1.0f / __builtin_sqrtf(sum_rows(kk) + kNormEps);
      rqn = a.scale / __builtin_sqrtf(sum_rows(qq) + kNormEps);
    }
    const float be = DELTA ? a.beta[t * a.ld_beta + h] : 1.0f;
    f32x4 u;
    u16x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = bf16_value(vr[j]);
      if constexpr (DELTA) u[j] = be * (u[j] - al * (rk * sum_rows(ks[j])));
      u[j] *= rk;                     // the key's norm goes with u into k u^T
      o[j] = bf16_bits(rqn * __builtin_fmaf(kq, u[j], al * sum_rows(qs[j])));
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = __builtin_fmaf(kv[i], u[j], al * s[i][j]);
    if (lane < 4)
      *reinterpret_cast<u16x4*>(a.out + t * a.out_token + h * a.out_head + col * 2) = o;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) *reinterpret_cast<f32x4*>(sp + i * a.dv) = s[i];
}

GdnArgs args_of(const GdnCall& c) {
  GdnArgs a = {};
  a.q = static_cast<const uint8_t*>(c.q.p);
  a.k = static_cast<const uint8_t*>(c.k.p);
  a.v = static_cast<const uint8_t*>(c.v.p);
  a.q_token = c.q.token * 2; a.q_head = c.q.head * 2;
  a.k_token = c.k.token * 2; a.k_head = c.k.head * 2;
  a.v_token = c.v.token * 2; a.v_head = c.v.head * 2;
  a.alpha = c.alpha; a.beta = c.beta; a.ld_alpha = c.ld_alpha; a.ld_beta = c.ld_beta;
  a.out = static_cast<uint8_t*>(c.out);
  a.out_token = c.out_token * 2; a.out_head = c.out_head * 2;
  a.state = c.state; a.n_slots = c.n_slots; a.slot_stride = c.slot_stride;
  a.slots = c.slots; a.cu = c.cu; a.cached = c.cached;
  a.n_tokens = static_cast<int>(c.n_tokens); a.n_requests = static_cast<int>(c.n_requests);
  a.n_heads = static_cast<int>(c.n_heads); a.group = static_cast<int>(c.n_heads / c.n_k_heads);
  a.dv = static_cast<int>(c.dv); a.scale = c.scale; a.normalize = c.normalize;
  return a;
}

template <int DK>
void launch_tokens(const GdnArgs& a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.n_requests) * a.n_heads *
                                              ((a.dv + 63) / 64));
  if (a.beta) gdn_tokens_kernel<DK, true><<<grid, 256, 0, stream>>>(a);
  else gdn_tokens_kernel<DK, false><<<grid, 256, 0, stream>>>(a);
}

}  // namespace

int64_t gdn_workspace(const GdnCall&) { return 0; }

hipError_t launch_gdn(const GdnCall& c, hipStream_t stream) {
  if (c.n_tokens == 0) return hipSuccess;
  const GdnArgs a = args_of(c);
  if (c.dk == 64) launch_tokens<64>(a, stream);
  else launch_tokens<128>(a, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
