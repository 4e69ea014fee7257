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
// A column of S depends on no other column, so a wave owns 16 or 32 columns and
// all rows, and nothing is exchanged between waves.  The state passes once in and
// once out, whatever the tokens in between; for single tokens that is all there
// is to move, and the kernel is bound by it.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "gemm_common.h"
#include "internal.h"

namespace nvfp4 {
namespace {

typedef unsigned short u16x4 __attribute__((ext_vector_type(4)));
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
  int few;                            // requests of at most so many tokens go token after token
  int share, parts;                   // items of a part of a key head's, parts
  uint8_t* records;                   // of chunks and heads
  float* decays;                      // of whole chunks
};

__device__ __forceinline__ float bf16_value(unsigned short x) {
  return __uint_as_float(static_cast<unsigned>(x) << 16);
}

__device__ __forceinline__ unsigned short bf16_bits(float f) {
  return __builtin_bit_cast(unsigned short, static_cast<__bf16>(f));
}

// Sum over the lanes that share lane % LC; every one of them gets it.
template <int LC>
__device__ __forceinline__ float sum_rows(float x) {
  if constexpr (LC <= 2)
    x += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x122, 0xF, 0xF, false));
  if constexpr (LC <= 4)
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

// Token after token.  Lane l has the four columns from 4 (l % LC) of its wave's 4 LC
// and the dk LC / 64 rows from there times l / LC.
//
// Bound by reading and writing the states: 32 requests of one token, 64 heads of
// 128 x 128 (268 MB): 44.6 us, 6.0 TB/s.  Waves of 16 columns, which ask for half
// lines: 57.3 -> 52.9 us; states written past the caches, where they would take
// the place of what the next layer reads: 52.9 -> 44.6.
template <int DK, bool DELTA, int LC>
__device__ __forceinline__ void few_tokens(const GdnArgs& a, int wave) {
  constexpr int R = DK / 64 * LC;
  const int lane = threadIdx.x & 63;
  const int slices = (a.dv + 4 * LC - 1) / (4 * LC), rh = wave / slices;
  const int col = (wave - rh * slices) * 4 * LC + lane % LC * 4;
  const int r = rh / a.n_heads, h = rh - r * a.n_heads, hk = h / a.group;
  if (r >= a.n_requests || col >= a.dv) return;
  const Request rq = request_of(a, r);
  if (rq.len < 1 || rq.len > a.few) return;
  const int row0 = lane / LC * R;
  float* sp = a.state + rq.slot * a.slot_stride + (static_cast<int64_t>(h) * DK + row0) * a.dv + col;
  f32x4 s[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    s[i] = rq.fresh ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : *reinterpret_cast<const f32x4*>(sp + i * a.dv);
  // a token's inputs, asked for while the one before is computed
  typedef unsigned short row_t __attribute__((ext_vector_type(R)));
  struct Token {
    row_t k, q;
    u16x4 v;
    float alpha, beta;
  };
  auto token = [&](int t) __attribute__((always_inline)) {
    return Token{*reinterpret_cast<const row_t*>(a.k + t * a.k_token + hk * a.k_head + row0 * 2),
                 *reinterpret_cast<const row_t*>(a.q + t * a.q_token + hk * a.q_head + row0 * 2),
                 *reinterpret_cast<const u16x4*>(a.v + t * a.v_token + h * a.v_head + col * 2),
                 a.alpha[t * a.ld_alpha + h], DELTA ? a.beta[t * a.ld_beta + h] : 1.0f};
  };
  const int end = rq.first + rq.len;
  Token next = token(rq.first);
  for (int t = rq.first; t < end; ++t) {
    const Token now = next;
    if (t + 1 < end) next = token(t + 1);
    const row_t kr = now.k, qr = now.q;
    const u16x4 vr = now.v;
    const float al = now.alpha, be = now.beta;
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
    kq = sum_rows<LC>(kq);
    float rk = 1.0f, rqn = a.scale;
    if (a.normalize) {
      rk = 1.0f / __builtin_sqrtf(sum_rows<LC>(kk) + kNormEps);
      rqn = a.scale / __builtin_sqrtf(sum_rows<LC>(qq) + kNormEps);
    }
    f32x4 u;
    u16x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = bf16_value(vr[j]);
      if constexpr (DELTA) u[j] = be * (u[j] - al * (rk * sum_rows<LC>(ks[j])));
      u[j] *= rk;                     // the key's norm goes with u into k u^T
      o[j] = bf16_bits(rqn * __builtin_fmaf(kq, u[j], al * sum_rows<LC>(qs[j])));
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = __builtin_fmaf(kv[i], u[j], al * s[i][j]);
    if (lane < LC)
      *reinterpret_cast<u16x4*>(a.out + t * a.out_token + h * a.out_head + col * 2) = o;
  }
#pragma unroll
  for (int i = 0; i < R; ++i) __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(sp + i * a.dv));
}

template <int DK, bool DELTA, int LC>
__global__ void __launch_bounds__(256)
gdn_tokens_kernel(const GdnArgs a) {
  few_tokens<DK, DELTA, LC>(a, __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6)));
}

// ---------------------------------------------------------------------------
// Chunks of 64 tokens.
//
// With g_i the product of the decays up to token i of a chunk and S0 the state
// before it,
//   (1 + A) U = diag(beta) (V - diag(g) K S0),  A_ij = beta_i g_i/g_j k_i.k_j, j < i
//   O = scale (diag(g) Q S0 + P U),             P_ij = g_i/g_j q_i.k_j, j <= i
//   S = g_64 S0 + K^T diag(g_64 / g_j) U
// (plain rule: U = V).  What does not depend on the state is made for all chunks
// at once by prepare_kernel: T = (1 + A)^-1 diag(beta), P and the factors of rows,
// a record of a chunk and head.  Then scan_kernel goes through a request's chunks
// in order with the products that do: K S0, T R, Q S0, P U, K^T U.
//
// A wave of scan_kernel owns 16 columns of S, U and O and all their rows.  With
// rows down and columns across lanes, the sums of one product (lane l: column
// l % 16, four rows of a tile of 16 from 4 (l / 16)) are the right operand of
// the next as they are, if the tiles' rows are taken in this order: tile 2 s + e,
// row 4 g + i is row 32 s + 8 g + 4 e + i, so that a lane's eight values of two
// tiles are the eight of a k-step of 32.  So nothing passes between lanes or
// waves, and only left operands (K, Q, K^T, T, P) are read from LDS.
//
// Precision.  K, Q and V are bf16, so products with them are exact; norms,
// decays, beta and the scale are factors of rows in binary32.  S, U, R and T are
// binary32 and enter products as sums of bf16 numbers: S and T two (16 bits), R
// and U into the state three (24), the diagonal of T none at all.  R in two and
// without its second part's product with T's: the scan of 32768 tokens 6 % shorter,
// the state's error (2-norm, 0.1 to 1.8e-6) 1.5 times as large; S in three: 11 % longer
// and 0.7 times.  Outputs take S, P and U in two, which leaves them their own rounding
// to bf16 (1.66e-3 in the 2-norm; with S and P in one number each 2.3 to 2.5e-3, and the
// scan of 32768 tokens 960 us instead of 1000).  Decays are added up as base-2
// logarithms in binary64, so that a gate close to zero takes nothing from the others.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int kChunk = 64;
// A record: the lower triangles of T and of P (high and low parts, six operands of
// 1 KB each), and four factors of each row.  Operand index of the tile of rows t and
// the k-step s <= t / 2.
__device__ __forceinline__ constexpr int tri(int t, int s) { return t < 2 ? t : 2 * t - 2 + s; }
template <bool DELTA>
struct Record {
  static constexpr int kT = 0;                               // high, then low
  static constexpr int kP = DELTA ? 12 * 1024 : 0;
  static constexpr int kRows = kP + 12 * 1024;               // a, b, c, beta: 64 floats each
  static constexpr int kBytes = kRows + 1024;
};

__device__ __forceinline__ unsigned pack_bf16(float x, float y) {
  const bf16x2 p = {static_cast<__bf16>(x), static_cast<__bf16>(y)};
  return __builtin_bit_cast(unsigned, p);
}
// x and y less the two bf16 numbers that p holds
__device__ __forceinline__ void less_bf16(float* x, float* y, unsigned p) {
  *x -= __uint_as_float(p << 16);
  *y -= __uint_as_float(p & 0xFFFF0000u);
}

// Eight binary32 numbers as sums of N bf16 ones.
template <int N>
struct Parts {
  u32x4 p[N];
  __device__ __forceinline__ void of(f32x4 x, f32x4 y) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        unsigned u = pack_bf16(x[2 * i], x[2 * i + 1]), w = pack_bf16(y[2 * i], y[2 * i + 1]);
        // opaque, or the compiler rounds each number again to take it off
        if (n + 1 < N) asm("" : "+v"(u), "+v"(w));
        p[n][i] = u;
        p[n][2 + i] = w;
        if (n + 1 < N) {
          float x0 = x[2 * i], x1 = x[2 * i + 1], y0 = y[2 * i], y1 = y[2 * i + 1];
          less_bf16(&x0, &x1, u);
          less_bf16(&y0, &y1, w);
          x[2 * i] = x0; x[2 * i + 1] = x1; y[2 * i] = y0; y[2 * i + 1] = y1;
        }
      }
    }
  }
};

__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// 2^d for d <= 0 in binary64, to binary32's precision
__device__ __forceinline__ float exp2_of(double d) {
  const double n = __builtin_rint(d);
  const int e = n < -1000.0 ? -1000 : static_cast<int>(n);
  return __builtin_ldexpf(__builtin_amdgcn_exp2f(static_cast<float>(d - n)), e);
}

// First chunk slot of request r: floor(rows before / 64) + r leaves every
// request at least the chunks that it fills, without a prefix sum of its own.
__device__ __forceinline__ int first_slot(const GdnArgs& a, int r) {
  const int row = min(max(a.cu[r], 0), a.n_tokens);
  return row / kChunk + r;
}

// The request that chunk slot t belongs to, the last r with first_slot(r) <= t;
// -1 if there is none.  Each round the wave's 64 lanes probe 64 places.
__device__ __forceinline__ int request_at(const GdnArgs& a, int t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = a.n_requests;
  for (bool first = true; n > 1 || first; first = false) {
    const int step = (n + 63) >> 6;
    const bool ok = lane * step < n && first_slot(a, lo + lane * step) <= t;
    const int count = __popcll(__ballot(ok));
    if (count == 0) return -1;
    lo += (count - 1) * step;
    n = min(step, n - (count - 1) * step);
  }
  return lo;
}

// Rows of [64][DK] bf16 in LDS: 16-byte pieces exchanged by an exclusive or.
template <int DK>
struct Rows {
  static constexpr int kBytes = DK * 2, kPieces = DK / 8;
  // 16 lanes with consecutive rows, or with rows 0-3, 8-11, 16-19, 24-27
  // (+ 4), fall on different banks
  __device__ static __forceinline__ int natural(int row) { return row & (kPieces - 1); }
  __device__ static __forceinline__ int paired(int row) {
    return DK == 128 ? (row & 3) | (((row >> 3) & 3) << 2) : ((row >> 1) & 1) | (((row >> 3) & 3) << 1);
  }
};

// One chunk and key head a workgroup: products of its keys and queries, then a
// value head a wave.
//
// Decays between tokens of different blocks of 16 are products of two factors,
// from the one to the start of the other's block and from there: both at most 1,
// so neither overflows, and few exponentials are left (D_ij = e_i f_j; within a
// block each has its own).  The inverse is taken in blocks of 16: those on the
// diagonal by substitution, a column a lane, the others by products in binary32
// (T_ij = - T_ii sum_m A_im T_mj), so no bit is lost to powers of A where keys
// resemble each other.
//
// What it waits for bounds it.  32768 tokens, 16 key and 64 value heads of 128
// (1.1 GB read and written): 254 us, 4.3 TB/s (238 with P in one part).  Before a
// workgroup brought the next unit's K and Q and gates while it works on one it took
// 1.3 times as long: the inverses 0.35 of it, K and Q 0.31 and T's stores 0.15.
constexpr int kPad = 68;                 // row of 64 floats in LDS
template <int DK, bool DELTA, int WAVES>
struct PrepareLds {
  static constexpr int kStage = 2 * kChunk * DK * 2, kProducts = (DELTA ? 2 : 1) * kChunk * kPad * 4;
  static constexpr int kShared = kStage > kProducts ? kStage : kProducts;
  struct Wave {
    float rows[32 * kPad];               // T's or P's, 32 at a time
    double g[kChunk];                    // logarithms of the decays up to each token
    float e[kChunk], f[3][kChunk];       // factors of rows; of columns, for blocks 1 to 3
    float beta[kChunk];
  };
  alignas(16) uint8_t shared[kShared];
  alignas(16) Wave wave[WAVES];
  alignas(16) float rk[kChunk], rq[kChunk];
};

// 32 rows of T or P from LDS (buf, of tiles 2 half and 2 half + 1) as left
// operands
template <class F>
__device__ __forceinline__ void operand_rows(const float* buf, int half, F&& put) {
  const int lr = threadIdx.x & 15, g4 = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int in = 8 * (lr >> 2) + 4 * e + (lr & 3);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s > half) continue;
      const int col = 32 * s + 8 * g4;
      put(2 * half + e, s, 32 * half + in, col,
          *reinterpret_cast<const f32x4*>(buf + in * kPad + col),
          *reinterpret_cast<const f32x4*>(buf + in * kPad + col + 4));
    }
  }
}

template <int DK, bool DELTA, int WAVES>
__global__ void __launch_bounds__(WAVES * 64, WAVES == 4 ? 2 : 1)
prepare_kernel(const GdnArgs a, int k_heads, int units, int workgroups) {
  // The workgroups behind those of the preparation take the requests of few tokens,
  // whose states come from memory while the others compute (3 prompts and 21 single
  // tokens, 48 heads: 29 us, one after the other 38).
  if (static_cast<int>(blockIdx.x) >= workgroups) {
    few_tokens<DK, DELTA, 8>(a, __builtin_amdgcn_readfirstlane((blockIdx.x - workgroups) * WAVES +
                                                            (threadIdx.x >> 6)));
    return;
  }
  using L = Rows<DK>;
  using Rec = Record<DELTA>;
  __shared__ PrepareLds<DK, DELTA, WAVES> lds;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int lr = lane & 15, g4 = lane >> 4;

  // Of a unit (a chunk slot and key head) a thread brings pieces of K and Q and a
  // lane's gates of its wave's first head; len 0: nothing to do there.
  constexpr bool kAhead = WAVES == 4;
  constexpr int kLoads = 2 * kChunk * L::kPieces / (WAVES * 64);
  struct Unit {
    int slot, hk, len;
    int64_t t0;
  };
  auto unit_at = [&](int i) {
    Unit u = {0, 0, 0, 0};
    if (i >= units) return u;
    u.slot = i / k_heads;
    u.hk = i - u.slot * k_heads;
    const int r = request_at(a, u.slot);
    if (r < 0) return u;
    const Request rq = request_of(a, r);
    const int c = u.slot - first_slot(a, r);
    if (rq.len <= a.few || c < 0 || c * kChunk >= rq.len) return u;
    u.len = min(rq.len - c * kChunk, kChunk);
    u.t0 = rq.first + static_cast<int64_t>(c) * kChunk;
    return u;
  };
  u32x4 x[kLoads];
  float gate, be;
  auto gates = [&](const Unit& u, int hh) __attribute__((always_inline)) {
    gate = 1.0f;
    be = 0.0f;
    if (lane < u.len && hh < a.group) {
      gate = a.alpha[(u.t0 + lane) * a.ld_alpha + u.hk * a.group + hh];
      if (DELTA) be = a.beta[(u.t0 + lane) * a.ld_beta + u.hk * a.group + hh];
    }
  };
  auto rows = [&](const Unit& u) __attribute__((always_inline)) {
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int i = n * WAVES * 64 + threadIdx.x;
      const int row = (i / L::kPieces) & (kChunk - 1), piece = i & (L::kPieces - 1);
      const uint8_t* p = i >= kChunk * L::kPieces ? a.q + (u.t0 + row) * a.q_token + u.hk * a.q_head
                                                  : a.k + (u.t0 + row) * a.k_token + u.hk * a.k_head;
      x[n] = u32x4{0u, 0u, 0u, 0u};
      if (row < u.len) x[n] = *reinterpret_cast<const u32x4*>(p + piece * 16);
    }
  };
  Unit next = unit_at(blockIdx.x);
  gates(next, wave);
  rows(next);
  int i = blockIdx.x;
  do {
    const Unit u = next;
    next = unit_at(kAhead ? i + workgroups : units);
    const int slot = u.slot, hk = u.hk, len = u.len;
    const int64_t t0 = u.t0;
    if (len == 0) {
      if (!kAhead) return;
      gates(next, wave);
      rows(next);
      continue;
    }

    // K and Q to LDS, when everybody has done with the unit before
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int i = n * WAVES * 64 + threadIdx.x;
      const int row = (i / L::kPieces) & (kChunk - 1), piece = i & (L::kPieces - 1);
      *reinterpret_cast<u32x4*>(lds.shared + (i >= kChunk * L::kPieces ? kChunk * L::kBytes : 0) +
                                row * L::kBytes + (piece ^ L::natural(row)) * 16) = x[n];
    }
    __syncthreads();
    if (kAhead) rows(next);
    auto at = [&](int is_q, int tile, int s) {
      const int row = tile * 16 + lr;
      return *reinterpret_cast<const u32x4*>(lds.shared + is_q * kChunk * L::kBytes + row * L::kBytes +
                                             ((4 * s + g4) ^ L::natural(row)) * 16);
    };
    // products of a tile of rows with the tiles of keys up to it; they stay in
    // registers until everybody has read K and Q
    constexpr int kTiles = 4 / WAVES;
    f32x4 kk[kTiles][4], qk[kTiles][4], qq[kTiles];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int t = wave + n * WAVES;
      qq[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < 4; ++u) kk[n][u] = qk[n][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) {
        const u32x4 ka = at(0, t, s), qa = at(1, t, s);
        qq[n] = mma(qa, qa, qq[n]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (u <= t) {
            const u32x4 kb = at(0, u, s);
            if (DELTA || u == t) kk[n][u] = mma(ka, kb, kk[n][u]);
            qk[n][u] = mma(qa, kb, qk[n][u]);
          }
      }
    }
    __syncthreads();
    float* const qkp = reinterpret_cast<float*>(lds.shared);
    float* const kkp = qkp + kChunk * kPad;
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int t = wave + n * WAVES;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (u <= t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (DELTA) kkp[(t * 16 + 4 * g4 + i) * kPad + u * 16 + lr] = kk[n][u][i];
            qkp[(t * 16 + 4 * g4 + i) * kPad + u * 16 + lr] = qk[n][u][i];
            if (u == t && 4 * g4 + i == lr) {
              lds.rk[t * 16 + lr] = kk[n][u][i];
              lds.rq[t * 16 + lr] = qq[n][i];
            }
          }
    }
    __syncthreads();
    if (wave == 0) {
      lds.rk[lane] = a.normalize ? 1.0f / __builtin_sqrtf(lds.rk[lane] + kNormEps) : 1.0f;
      lds.rq[lane] = a.normalize ? a.scale / __builtin_sqrtf(lds.rq[lane] + kNormEps) : a.scale;
    }
    __syncthreads();

    auto& own = lds.wave[wave];
    float* const buf = own.rows;
    for (int hh = wave; hh < a.group; hh += WAVES) {
      const int h = hk * a.group + hh;
      // a gate of zero counts as 2^-160, below what binary32 holds
      double sum = gate > 0.0f ? log2(static_cast<double>(gate)) : gate == 0.0f ? -160.0 : __builtin_nan("");
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double before = __shfl_up(sum, d);
        if (lane >= d) sum += before;
      }
      const double last = __shfl(sum, 63);
      uint8_t* const rec = a.records + (static_cast<int64_t>(slot) * a.n_heads + h) * Rec::kBytes;
      {
        const float rk = lds.rk[lane], gi = exp2_of(sum);
        float* const rows = reinterpret_cast<float*>(rec + Rec::kRows);
        rows[lane] = gi * rk;
        rows[64 + lane] = gi * lds.rq[lane];
        rows[128 + lane] = rk * exp2_of(last - sum);
        if (DELTA) rows[192 + lane] = be;
        if (lane == 0) a.decays[static_cast<int64_t>(slot) * a.n_heads + h] = exp2_of(last);
        own.g[lane] = sum;
        own.beta[lane] = be;
        // asked for before the work on this head
        if (hh + WAVES < a.group) gates(u, hh + WAVES);
        else if (kAhead) gates(next, wave);
        own.e[lane] = exp2_of(sum - __shfl(sum, lane & 48));
#pragma unroll
        for (int b = 1; b < 4; ++b) {
          const double start = __shfl(sum, 16 * b);
          own.f[b - 1][lane] = lane < 16 * b ? rk * exp2_of(start - sum) : 0.0f;
        }
      }
      __builtin_amdgcn_wave_barrier();

      // decays times the columns' norms of tile (i, m), of row i 16 + lr, columns
      // m 16 + 4 g4 + 0 .. 3
      f32x4 within[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double gi = own.g[i * 16 + lr];
        const f32x4 rk = *reinterpret_cast<const f32x4*>(lds.rk + i * 16 + 4 * g4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          within[i][e] = 4 * g4 + e <= lr ? rk[e] * exp2_of(gi - own.g[i * 16 + 4 * g4 + e]) : 0.0f;
      }
      auto decay = [&](int i, int m) {
        if (i == m) return within[i];
        return own.e[i * 16 + lr] * *reinterpret_cast<const f32x4*>(&own.f[i - 1][m * 16 + 4 * g4]);
      };

      if constexpr (DELTA) {
        // -A: tiles below the diagonal as left operands, those on it in LDS
        f32x4 na[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = i * 16 + lr;
          const float f = -own.beta[row] * lds.rk[row];
#pragma unroll
          for (int m = 0; m <= i; ++m) {
            na[i][m] = f * decay(i, m) * *reinterpret_cast<const f32x4*>(kkp + row * kPad + m * 16 + 4 * g4);
            if (m == i)
#pragma unroll
              for (int e = 0; e < 4; ++e) na[i][i][e] = 4 * g4 + e < lr ? na[i][i][e] : 0.0f;
          }
          *reinterpret_cast<f32x4*>(buf + row * 20 + 4 * g4) = na[i][i];
        }
        __builtin_amdgcn_wave_barrier();
        // the diagonal blocks' inverses: lane l has column l % 16 of block l / 16
        float x[16];
#pragma unroll
        for (int row = 0; row < 16; ++row) {
          float y = row == lr ? 1.0f : 0.0f;
#pragma unroll
          for (int m = 0; m < row; m += 4) {
            const f32x4 w = *reinterpret_cast<const f32x4*>(buf + (g4 * 16 + row) * 20 + m);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (m + e < row) y = __builtin_fmaf(w[e], x[m + e], y);
          }
          x[row] = y;
        }
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int row = 0; row < 16; ++row) buf[(g4 * 16 + row) * 20 + lr] = x[row];
        __builtin_amdgcn_wave_barrier();
        f32x4 dl[4], t[4][4];              // as left operands; tiles of the inverse
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dl[i] = *reinterpret_cast<const f32x4*>(buf + (i * 16 + lr) * 20 + 4 * g4);
#pragma unroll
          for (int e = 0; e < 4; ++e) t[i][i][e] = buf[(i * 16 + 4 * g4 + e) * 20 + lr];
        }
        __builtin_amdgcn_wave_barrier();
        auto times = [](f32x4 left, f32x4 right, f32x4 acc) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(left[e], right[e], acc, 0, 0, 0);
          return acc;
        };
#pragma unroll
        for (int d = 1; d < 4; ++d)
#pragma unroll
          for (int j = 0; j + d < 4; ++j) {
            const int i = j + d;
            f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int m = j; m < i; ++m) acc = times(na[i][m], t[m][j], acc);
            t[i][j] = times(dl[i], acc, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
          }
        // 32 rows at a time through LDS to the operands' order, times beta,
        // below the diagonal only
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2 * half + 2; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                buf[(i * 16 + 4 * g4 + e) * kPad + j * 16 + lr] = j <= 2 * half + i ? t[2 * half + i][j][e] : 0.0f;
          __builtin_amdgcn_wave_barrier();
          operand_rows(buf, half, [&](int tile, int s, int row, int col, f32x4 y0, f32x4 y1) {
            y0 *= *reinterpret_cast<const f32x4*>(own.beta + col);
            y1 *= *reinterpret_cast<const f32x4*>(own.beta + col + 4);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              y0[q] = col + q < row ? y0[q] : 0.0f;
              y1[q] = col + 4 + q < row ? y1[q] : 0.0f;
            }
            Parts<2> w;
            w.of(y0, y1);
            uint8_t* const dst = rec + Rec::kT + tri(tile, s) * 1024 + lane * 16;
            *reinterpret_cast<u32x4*>(dst) = w.p[0];
            *reinterpret_cast<u32x4*>(dst + 6 * 1024) = w.p[1];
          });
          __builtin_amdgcn_wave_barrier();
        }
      }
      // P, the same way
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = (2 * half + i) * 16 + lr;
          const float f = lds.rq[row];
#pragma unroll
          for (int m = 0; m < 2 * half + 2; ++m) {
            f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
            if (m <= 2 * half + i)
              y = f * decay(2 * half + i, m) * *reinterpret_cast<const f32x4*>(qkp + row * kPad + m * 16 + 4 * g4);
            *reinterpret_cast<f32x4*>(buf + (i * 16 + lr) * kPad + m * 16 + 4 * g4) = y;
          }
        }
        __builtin_amdgcn_wave_barrier();
        operand_rows(buf, half, [&](int tile, int s, int, int, f32x4 y0, f32x4 y1) {
          Parts<2> w;
          w.of(y0, y1);
          uint8_t* const dst = rec + Rec::kP + tri(tile, s) * 1024 + lane * 16;
          *reinterpret_cast<u32x4*>(dst) = w.p[0];
          *reinterpret_cast<u32x4*>(dst + 6 * 1024) = w.p[1];
        });
        __builtin_amdgcn_wave_barrier();
      }
    }
  } while (kAhead && (i += workgroups) < units);
}

// The scan: 32 columns of a request's head are an item; a workgroup of five waves
// goes through the chunks of its items.
//
// What the next chunk waits for is the way from one state to the next, so that
// is all that the two state waves do, 16 columns each: K S0, R, U, K^T U.  The
// two output waves take Q S0 and then P U, from operands that a state wave leaves
// in LDS as it makes them.  The loader brings everything from memory to LDS, K, T
// and V two chunks ahead, also those of the next item.
//
// Barriers, two a chunk.  Behind the first of chunk c, its K, T, V and Q have
// landed, as has P of c - 1, and S0 of c and U of c - 1 are in LDS: the output
// waves take S0 to registers and finish c - 1 with P U.  Behind the second they have,
// and the state waves may write U of c and S0 of c + 1 over them and the loader P of c
// over that of c - 1; the state waves have read T and V of c, and the loader brings
// those of c + 2 there.  (P of two chunks where LDS holds them, dk 64 or the plain
// rule, and P U behind the second barrier: 2 to 5 % longer.)
//
// One prompt of 32768 tokens, 16 key and 64 value heads of 128 (an item on each
// CU): 1000 us, 2.0 a chunk.  The state waves bound it (782 of 962 were left without
// output and loader when S and P went to outputs, and R to U, in a part less): their
// 110 products a chunk take 370, the rest is what each waits for of the one before.
// The plain rule's state waves do little; there a chunk's loads bound it, 21 bytes a
// cycle to LDS (with P in one part, 43 KB instead of 49, it took 12 % less).
constexpr int kScanCols = 32, kRing = 3, kScanThreads = 320;
template <int DK, bool DELTA>
struct ScanLds {
  // of three chunks: K and the factors of rows
  static constexpr int kK = 0, kRows = kChunk * DK * 2, kIn = kRows + 1024;
  // of two: T and V, which a state wave has read when half a chunk is done; Q
  static constexpr int kT = 0, kV = DELTA ? 12 * 1024 : 0, kMid = kV + kChunk * kScanCols * 2;
  static constexpr int kQ = kChunk * DK * 2;
  // of one: P
  static constexpr int kP = 12 * 1024;
  // of each state wave: S0 (two parts, as operands), U (binary32, by tiles)
  static constexpr int kS = 0, kU = DK / 32 * 2048, kWave = kU + 4 * 1024;
};

// LDS by its own address space: with generic pointers the compiler joins the
// paths of the two places of a buffer and then tests the pointer for null.
#define NVFP4_LDS __attribute__((address_space(3)))
typedef NVFP4_LDS uint8_t lds_t;

template <class T>
__device__ __forceinline__ T lds_read(const lds_t* p) {
  return *(const NVFP4_LDS T*)(p);
}
__device__ __forceinline__ void lds_write(lds_t* p, u32x4 x) { *(NVFP4_LDS u32x4*)(p) = x; }

__device__ __forceinline__ s16x4 read_tr(const lds_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((NVFP4_LDS s16x4*)(p));
}

// 16 bytes a lane straight to LDS at lds + 16 * lane
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t rsrc, lds_t* lds, unsigned off) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (NVFP4_LDS void*)lds, 16, off, 0, 0, 0);
#endif
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const uint8_t* base, unsigned bytes = 0x7FFFFFFF) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  const unsigned lo = __builtin_amdgcn_readfirstlane(static_cast<unsigned>(p));
  const unsigned hi = __builtin_amdgcn_readfirstlane(static_cast<unsigned>(p >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(
      reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0, bytes, 0x00020000);
}

// A request's head and columns; chunks 0: none.
struct Scan {
  Request rq;
  int h, hk, slice, chunks;
  int64_t slot0;
};

constexpr unsigned kOutside = 0x80000000u;         // of the resources' range

// The loader's loads to LDS.  It always makes the same number of them (rows and
// chunks past the end read as zeros), which its waits count.
template <int DK, bool DELTA>
struct ScanLoads {
  using L = Rows<DK>;
  using Lds = ScanLds<DK, DELTA>;
  using Rec = Record<DELTA>;
  static constexpr int kRowLoads = kChunk * DK * 2 / 1024, kValues = kChunk * kScanCols * 2 / 1024;
  static constexpr int kIn = kRowLoads + (DELTA ? 12 : 0) + 1 + kValues;

  static __device__ __forceinline__ void rows(const uint8_t* base, int64_t stride, int len, lds_t* lds) {
    const __amdgpu_buffer_rsrc_t rsrc = resource(base);
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int n = 0; n < kRowLoads; ++n) {
      const int at = n * 64 + lane;
      const int row = at / L::kPieces, piece = (at & (L::kPieces - 1)) ^ L::paired(row);
      load_lds(rsrc, lds + n * 1024,
               row < len ? static_cast<unsigned>(row * stride) + piece * 16 : kOutside);
    }
  }
  // K and the factors of rows of chunk c to `lds`, T and V to `mid`
  static __device__ __forceinline__ void in(const GdnArgs& a, const Scan& w, int c, lds_t* lds,
                                            lds_t* mid) {
    const int lane = threadIdx.x & 63;
    const bool real = c < w.chunks;
    const int len = real ? min(w.rq.len - c * kChunk, kChunk) : 0;
    const int64_t t0 = w.rq.first + static_cast<int64_t>(real ? c : 0) * kChunk;
    rows(a.k + t0 * a.k_token + w.hk * a.k_head, a.k_token, len, lds + Lds::kK);
    const __amdgpu_buffer_rsrc_t vr = resource(a.v + t0 * a.v_token + w.h * a.v_head);
    const __amdgpu_buffer_rsrc_t rec =
        resource(a.records + ((w.slot0 + (real ? c : 0)) * a.n_heads + w.h) * Rec::kBytes);
    if constexpr (DELTA)
#pragma unroll
      for (int n = 0; n < 12; ++n)
        load_lds(rec, mid + Lds::kT + n * 1024, real ? Rec::kT + n * 1024 + lane * 16 : kOutside);
    load_lds(rec, lds + Lds::kRows, real ? Rec::kRows + lane * 16 : kOutside);
#pragma unroll
    for (int n = 0; n < kValues; ++n) {
      const int at = n * 64 + lane;
      const int row = at / (kScanCols / 8), col = w.slice * kScanCols + at % (kScanCols / 8) * 8;
      load_lds(vr, mid + Lds::kV + n * 1024,
               row < len && col < a.dv ? static_cast<unsigned>(row * a.v_token) + col * 2 : kOutside);
    }
  }
  static __device__ __forceinline__ void q(const GdnArgs& a, const Scan& w, int c, lds_t* lds) {
    const bool real = c < w.chunks;
    const int len = real ? min(w.rq.len - c * kChunk, kChunk) : 0;
    const int64_t t0 = w.rq.first + static_cast<int64_t>(real ? c : 0) * kChunk;
    rows(a.q + t0 * a.q_token + w.hk * a.q_head, a.q_token, len, lds);
  }
  static __device__ __forceinline__ void p(const GdnArgs& a, const Scan& w, int c, lds_t* lds) {
    const bool real = c < w.chunks;
    const __amdgpu_buffer_rsrc_t rec =
        resource(a.records + ((w.slot0 + (real ? c : 0)) * a.n_heads + w.h) * Rec::kBytes);
#pragma unroll
    for (int n = 0; n < 12; ++n)
      load_lds(rec, lds + n * 1024,
               real ? Rec::kP + n * 1024 + (threadIdx.x & 63) * 16 : kOutside);
  }
};

// Four factors of the rows of tile t, the `which`-th of each
__device__ __forceinline__ f32x4 row_factors(const lds_t* lds, int which, int t) {
  const int g4 = (threadIdx.x & 63) >> 4;
  return lds_read<f32x4>(lds + 256 * which + (32 * (t / 2) + 8 * g4 + 4 * (t % 2)) * 4);
}

// Left operand of tile t, k-step s, of [64][DK] rows
template <int DK>
__device__ __forceinline__ u32x4 left_rows(const lds_t* lds, int t, int s) {
  const int lr = threadIdx.x & 15, g4 = (threadIdx.x & 63) >> 4;
  const int row = 32 * (t / 2) + 4 * (t % 2) + 8 * (lr >> 2) + (lr & 3);
  return lds_read<u32x4>(lds + row * Rows<DK>::kBytes + ((4 * s + g4) ^ Rows<DK>::paired(row)) * 16);
}

__device__ __forceinline__ u32x4 operand_at(const lds_t* lds, int n) {
  return lds_read<u32x4>(lds + n * 1024 + (threadIdx.x & 63) * 16);
}

// K^T operand of state tile t: its rows, tokens 32 s + 8 g4 + 0 .. 7
template <int DK>
__device__ __forceinline__ u32x4 left_columns(const lds_t* k, int t, int s) {
  const int lr = threadIdx.x & 15, g4 = (threadIdx.x & 63) >> 4;
  const int piece = 4 * (t / 2) + (lr & 3);
  s16x4 w[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = 32 * s + 8 * g4 + 4 * e + (lr >> 2);
    w[e] = read_tr(k + row * Rows<DK>::kBytes + (piece ^ Rows<DK>::paired(row)) * 16 + 8 * (t % 2));
  }
  return __builtin_bit_cast(u32x4, __builtin_shufflevector(w[0], w[1], 0, 1, 2, 3, 4, 5, 6, 7));
}

// End of a scheduling region of a state wave: N products, between which go VALU
// operations and LDS reads of what comes next.  One wave a SIMD hides nothing
// under another, so its own operations have to lie under its products.
template <int N, int VALU, int READS>
__device__ __forceinline__ void region() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (VALU > 0) __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    if constexpr (READS > 0) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// A state wave: 16 columns of the state.  Tile t, element i is row 32 (t / 2) + 8
// g4 + 4 (t % 2) + i.  `x`: the state as right operands.
template <int DK, bool DELTA>
struct State {
  using Lds = ScanLds<DK, DELTA>;
  static constexpr int kTiles = DK / 16, kSteps = DK / 32;
  f32x4 st[kTiles];
  Parts<2> x[kSteps];

  __device__ __forceinline__ void parts(int from, int to) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      if (s >= from && s < to) x[s].of(st[2 * s], st[2 * s + 1]);
  }
  // what the output wave takes of the state
  __device__ __forceinline__ void leave(lds_t* xc) const {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int n = 0; n < 2; ++n)
        lds_write(xc + Lds::kS + (2 * s + n) * 1024 + (threadIdx.x & 63) * 16, x[s].p[n]);
  }

  // From the state before a chunk to the one after it; U goes to xc behind the
  // barrier.
  __device__ __forceinline__ void chunk(float decay, int wave, const lds_t* in, const lds_t* mid,
                                        lds_t* xc) {
    const int lane = threadIdx.x & 63, lr = lane & 15, g4 = lane >> 4;
    const lds_t* const rows = in + Lds::kRows;
    f32x4 u[4], v[4], factor[4], last[4];
    s16x4 vb[4];
    u32x4 kt[2][kTiles];
    auto values = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        vb[t] = read_tr(mid + Lds::kV + (32 * (t / 2) + 8 * g4 + 4 * (t % 2) + (lr >> 2)) * (kScanCols * 2) +
                        wave * 32 + (lr & 3) * 8);
    };
    auto columns = [&](int s) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t) kt[s][t] = left_columns<DK>(in + Lds::kK, t, s);
    };
    auto factors = [&](f32x4 (&f)[4], int which) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 4; ++t) f[t] = row_factors(rows, which, t);
    };
    if constexpr (DELTA) {
      u32x4 k[kSteps][4], hi[6], lo[6];
      f32x4 a[4], beta[4];
      auto keys = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int t = 0; t < 4; ++t) k[s][t] = left_rows<DK>(in + Lds::kK, t, s);
      };
      keys(0);
      keys(1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        if (s + 2 < kSteps) keys(s + 2);
        if (s == kSteps - 2) {
          values();
          factors(a, 0);
        }
        if (s == kSteps - 1) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            hi[tri(t, 0)] = operand_at(mid + Lds::kT, tri(t, 0));
            lo[tri(t, 0)] = operand_at(mid + Lds::kT, 6 + tri(t, 0));
          }
          factors(beta, 3);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int t = 0; t < 4; ++t) u[t] = mma(k[s][t], x[s].p[n], u[t]);
        if (s == kSteps - 2) region<8, 0, (kSteps > 2 ? 2 : 1)>();
        else if (s == kSteps - 1) region<8, 0, 2>();
        else region<8, 0, 1>();
      }
      // R, and beta R, to which the products with T below the diagonal go
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[t][i] = __builtin_fmaf(-a[t][i], u[t][i], bf16_value(static_cast<unsigned short>(vb[t][i])));
        u[t] = beta[t] * v[t];
      }
      Parts<3> r0, r1;
      r0.of(v[0], v[1]);
#pragma unroll
      for (int t = 2; t < 4; ++t) {
        hi[tri(t, 1)] = operand_at(mid + Lds::kT, tri(t, 1));
        lo[tri(t, 1)] = operand_at(mid + Lds::kT, 6 + tri(t, 1));
      }
      factors(factor, 2);
      __builtin_amdgcn_sched_barrier(0);
      r1.of(v[2], v[3]);
      columns(0);
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] = mma(hi[tri(t, 0)], r0.p[0], u[t]);
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] = mma(hi[tri(t, 0)], r0.p[1], u[t]);
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] = mma(lo[tri(t, 0)], r0.p[0], u[t]);
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] = mma(lo[tri(t, 0)], r0.p[1], u[t]);
#pragma unroll
      for (int t = 0; t < 4; ++t) u[t] = mma(hi[tri(t, 0)], r0.p[2], u[t]);
      region<20, 2, 2>();
#pragma unroll
      for (int t = 2; t < 4; ++t) u[t] = mma(hi[tri(t, 1)], r1.p[0], u[t]);
#pragma unroll
      for (int t = 2; t < 4; ++t) u[t] = mma(hi[tri(t, 1)], r1.p[1], u[t]);
#pragma unroll
      for (int t = 2; t < 4; ++t) u[t] = mma(lo[tri(t, 1)], r1.p[0], u[t]);
#pragma unroll
      for (int t = 2; t < 4; ++t) u[t] = mma(lo[tri(t, 1)], r1.p[1], u[t]);
#pragma unroll
      for (int t = 2; t < 4; ++t) u[t] = mma(hi[tri(t, 1)], r1.p[2], u[t]);
    } else {
      values();
      factors(factor, 2);
      columns(0);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) u[t][i] = bf16_value(static_cast<unsigned short>(vb[t][i]));
    }
    Parts<3> y0, y1;
    y0.of(u[0] * factor[0], u[1] * factor[1]);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) st[t] *= decay;
    if constexpr (DELTA) region<6, 10, 0>();
    // The output wave has taken S0 of this chunk and U of the one before; lgkmcnt(0):
    // the loader fills T and V, which this wave has read.
    __builtin_amdgcn_s_waitcnt(0xC07F);
    stage_barrier();
#pragma unroll
    for (int t = 0; t < 4; ++t)
      lds_write(xc + Lds::kU + t * 1024 + lane * 16, __builtin_bit_cast(u32x4, u[t]));
    columns(1);
    y1.of(u[2] * factor[2], u[3] * factor[3]);
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
      for (int t = 0; t < kTiles; ++t) st[t] = mma(kt[0][t], y0.p[n], st[t]);
    region<3 * kTiles, 2, 1>();
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
      for (int t = 0; t < kTiles / 2; ++t) st[t] = mma(kt[1][t], y1.p[n], st[t]);
    __builtin_amdgcn_sched_barrier(0);
    parts(0, kSteps / 2);
#pragma unroll
    for (int n = 0; n < 3; ++n)
#pragma unroll
      for (int t = kTiles / 2; t < kTiles; ++t) st[t] = mma(kt[1][t], y1.p[n], st[t]);
    region<3 * kTiles / 2, 4, 0>();
    parts(kSteps / 2, kSteps);
    leave(xc);
  }
};

// The requests of more than `few` tokens in their order, 64 at a time in a wave's
// lanes, so that finding the next one mostly reads nothing: a load would wait for
// those to LDS before it.
struct Long {
  Request mine;
  int base, before;                    // of the 64: the first, and those wanted before it

  __device__ __forceinline__ void start(const GdnArgs& a) {
    base = before = 0;
    take(a);
  }
  __device__ __forceinline__ void take(const GdnArgs& a) {
    const int r = base + static_cast<int>(threadIdx.x & 63);
    mine = request_of(a, min(r, a.n_requests - 1));
    if (r >= a.n_requests) mine.len = 0;
  }
  // The n-th and its number, len 0 if they are fewer; n does not decrease.
  __device__ __forceinline__ Request nth(const GdnArgs& a, int n, int* number) {
    const int lane = threadIdx.x & 63;
    for (;;) {
      const bool is = mine.len > a.few;
      const uint64_t all = __ballot(is);
      const int count = __popcll(all);
      if (n - before < count) {
        const int at = __builtin_ctzll(
            __ballot(is && __popcll(all & ((uint64_t(1) << lane) - 1)) == n - before));
        *number = base + at;
        return {__builtin_amdgcn_readlane(mine.first, at), __builtin_amdgcn_readlane(mine.len, at),
                __builtin_amdgcn_readlane(static_cast<int>(mine.slot), at),
                __builtin_amdgcn_readlane(mine.fresh, at) != 0};
      }
      if (base + 64 >= a.n_requests) return {0, 0, 0, false};
      before += count;
      base += 64;
      take(a);
    }
  }
};

// A wave's place in the chunks of its workgroup's items, one item behind the
// other: chunk c of `w`, `next` the item behind.
//
// The value heads of a key head and their slices, which share K, Q and V, run on
// one XCD and its L2; the key heads go over the XCDs in turn, in parts if there are
// fewer than 8 of them.  Only requests that are long enough count, so that few of
// them fill the card too.
struct Cursor {
  Scan w, next;
  Long requests;
  int c, item;

  __device__ __forceinline__ void look(const GdnArgs& a) {
    const int slices = (a.dv + kScanCols - 1) / kScanCols;
    const int per_request = a.n_heads / a.group * a.parts;
    const int at = item / a.share, unit = at * 8 + blockIdx.x % 8;
    const int n = unit / per_request, part = unit - n * per_request;
    int r = 0;
    next.rq = requests.nth(a, n, &r);
    next.hk = part / a.parts;
    const int of_head = part % a.parts * a.share + item - at * a.share;
    next.h = next.hk * a.group + of_head / slices;
    next.slice = of_head % slices;
    next.chunks = (next.rq.len + kChunk - 1) / kChunk;
    next.slot0 = next.rq.first / kChunk + r;
    item += gridDim.x / 8;
  }
  __device__ __forceinline__ void start(const GdnArgs& a) {
    item = blockIdx.x / 8;
    requests.start(a);
    look(a);
    w = next;
    c = 0;
  }
  __device__ __forceinline__ bool valid() const { return c < w.chunks; }
  // To the next chunk; true if that is another item's.  The item behind it is
  // looked for before the step that leaves it, where that holds up nobody.
  __device__ __forceinline__ bool step() {
    if (++c < w.chunks) return false;
    if (w.chunks == 0) return false;
    w = next;
    c = 0;
    return true;
  }
};

template <int DK>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t state_of(const GdnArgs& a, const Scan& w) {
  return resource(reinterpret_cast<const uint8_t*>(a.state + w.rq.slot * a.slot_stride +
                                                   static_cast<int64_t>(w.h) * DK * a.dv));
}

// Bounds of 512 for its 320: at most 256 registers.  More, which LDS would leave
// room for, lie where each use by VALU operations costs a copy (1376 -> 1248 us).
template <int DK, bool DELTA>
__global__ void __launch_bounds__(512)
scan_kernel(const GdnArgs a) {
  using Lds = ScanLds<DK, DELTA>;
  using Loads = ScanLoads<DK, DELTA>;
  __shared__ __attribute__((aligned(1024))) uint8_t in_[kRing * Lds::kIn], mid_[2 * Lds::kMid],
      q_[2 * Lds::kQ], p_[Lds::kP], xc_[2 * Lds::kWave];
  const int lane = threadIdx.x & 63, lr = lane & 15, g4 = lane >> 4;
  // 0, 1: state, 2, 3: output, 4: loader.  The first wave, with which the fifth
  // shares a SIMD, is not a state wave (1077 -> 1004 us).
  const int id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = id == 0 ? 2 : id < 3 ? id - 1 : id;
  lds_t* const in = (lds_t*)in_;
  lds_t* const mid = (lds_t*)mid_;
  lds_t* const queries = (lds_t*)q_;
  lds_t* const scores = (lds_t*)p_;
  lds_t* const xc = (lds_t*)xc_;
  Cursor at;
  at.start(a);
  int place = 0;
  if (wave < 2) {
    State<DK, DELTA> s;
    float of_64 = 0.0f;                            // decays of 64 chunks, one a lane
    for (int g = 0;; g ^= 1) {
      // the last slice may have one wave's columns only
      const int col = at.w.slice * kScanCols + wave * 16;
      const unsigned place_in = col < a.dv ? (8 * g4 * a.dv + col + lr) * 4 : kOutside;
      if (at.valid() && (at.c & 63) == 0) {
        const float* const decays = a.decays + at.w.slot0 * a.n_heads + at.w.h;
        if (at.c + lane < at.w.chunks) of_64 = decays[(at.c + lane) * static_cast<int64_t>(a.n_heads)];
      }
      if (at.valid() && at.c == 0) {
        const __amdgpu_buffer_rsrc_t state = state_of<DK>(a, at.w);
#pragma unroll
        for (int t = 0; t < DK / 16; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s.st[t][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                state, at.w.rq.fresh ? kOutside : place_in, (32 * (t / 2) + 4 * (t % 2) + i) * a.dv * 4, 0));
        at.look(a);
        s.parts(0, DK / 32);
        s.leave(xc + wave * Lds::kWave);
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);          // lgkmcnt(0): S0 and U are in LDS
      stage_barrier();
      if (!at.valid()) break;
      const float decay = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(of_64), at.c & 63));
      s.chunk(decay, wave, in + place * Lds::kIn, mid + g * Lds::kMid, xc + wave * Lds::kWave);
      place = place == kRing - 1 ? 0 : place + 1;
      if (at.c == at.w.chunks - 1) {
        const __amdgpu_buffer_rsrc_t state = state_of<DK>(a, at.w);
#pragma unroll
        for (int t = 0; t < DK / 16; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s.st[t][i]), state, place_in,
                                                  (32 * (t / 2) + 4 * (t % 2) + i) * a.dv * 4, 0);
      }
      at.step();
    }
    stage_barrier();
  } else if (wave < 4) {
    const lds_t* const from = xc + (wave - 2) * Lds::kWave;
    f32x4 o[4];
    int len = 0;                                   // rows of the chunk whose outputs o is
    const uint8_t* rows = a.out;
    bool mine = false;
    at.look(a);
    for (int g = 0;; g ^= 1) {
      // lgkmcnt(0): the loader fills the Q that was read last
      __builtin_amdgcn_s_waitcnt(0xC07F);
      stage_barrier();
      u32x4 s0[DK / 32][2];
#pragma unroll
      for (int s = 0; s < DK / 32; ++s)
#pragma unroll
        for (int n = 0; n < 2; ++n) s0[s][n] = operand_at(from + Lds::kS, 2 * s + n);
      if (len > 0) {
        f32x4 u[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) u[t] = __builtin_bit_cast(f32x4, operand_at(from + Lds::kU, t));
        // it ends with the rows that there are
        const __amdgpu_buffer_rsrc_t rsrc =
            resource(rows, mine ? static_cast<unsigned>(len * a.out_token) : 0);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          Parts<DELTA ? 2 : 1> y;                  // the plain rule's U is bf16
          y.of(u[2 * s], u[2 * s + 1]);
          u32x4 p[4][2];
#pragma unroll
          for (int t = 2 * s; t < 4; ++t)
#pragma unroll
            for (int n = 0; n < 2; ++n) p[t][n] = operand_at(scores, 6 * n + tri(t, s));
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < (DELTA && n == 0 ? 2 : 1); ++i)
#pragma unroll
              for (int t = 2 * s; t < 4; ++t) o[t] = mma(p[t][n], y.p[i], o[t]);
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 32 * (t / 2) + 8 * g4 + 4 * (t % 2) + i;
            __builtin_amdgcn_raw_buffer_store_b16(
                bf16_bits(o[t][i]), rsrc, static_cast<unsigned>(row * a.out_token) + lr * 2, 0, 0);
          }
      }
      // lgkmcnt(0): S0 and U are taken, which the state waves write over, and P, which
      // the loader fills
      __builtin_amdgcn_s_waitcnt(0xC07F);
      stage_barrier();
      if (!at.valid()) break;
      const lds_t* const q = queries + g * Lds::kQ;
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) {
        u32x4 x[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) x[t] = left_rows<DK>(q, t, s);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int t = 0; t < 4; ++t) o[t] = mma(x[t], s0[s][n], o[t]);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t] *= row_factors(in + place * Lds::kIn + Lds::kRows, 1, t);
      place = place == kRing - 1 ? 0 : place + 1;
      const int col = at.w.slice * kScanCols + (wave - 2) * 16;
      mine = col < a.dv;
      len = min(at.w.rq.len - at.c * kChunk, kChunk);
      rows = a.out + (at.w.rq.first + static_cast<int64_t>(at.c) * kChunk) * a.out_token +
             at.w.h * a.out_head + col * 2;
      if (at.step()) at.look(a);
    }
  } else {
    // two chunks, one and none behind `at`
    Scan w0 = at.w, w1;
    int c0 = 0, c1;
    Loads::q(a, at.w, 0, queries);
    Loads::in(a, at.w, 0, in, mid);
    if (at.w.chunks == 1) at.look(a);
    bool looked = at.w.chunks == 1;
    if (at.step()) looked = false;
    w1 = at.w;
    c1 = at.c;
    Loads::in(a, w1, c1, in + Lds::kIn, mid + Lds::kMid);
    if (!looked) at.look(a);
    if (at.step()) at.look(a);
    place = 2;
    for (int g = 0;; g ^= 1) {
      // but for K, T and V of the next chunk, all that was asked for has landed
      __builtin_amdgcn_s_waitcnt(kVmcntKeepOf(Loads::kIn));
      stage_barrier();
      Loads::q(a, w1, c1, queries + (g ^ 1) * Lds::kQ);
      // the rest is not needed that soon, and would hold up the second barrier
      // (plain rule, 7 prompts: 42 -> 37 us)
      stage_barrier();
      Loads::p(a, w0, c0, scores);
      Loads::in(a, at.w, at.c, in + place * Lds::kIn, mid + g * Lds::kMid);
      place = place == kRing - 1 ? 0 : place + 1;
      if (c0 >= w0.chunks) break;
      w0 = w1;
      c0 = c1;
      w1 = at.w;
      c1 = at.c;
      if (at.step()) at.look(a);
    }
    // nothing is on its way to LDS when it is released
    __builtin_amdgcn_s_waitcnt(0);
  }
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

// Workgroups of the scan, one a CU, which go on to further items without a pause.
// 32 requests of 21 to 64 tokens, 64 heads of 128 x 128 (32 items a workgroup): 135
// to 149 us in all; 441 where each item began anew (before the lengths were kept in
// lanes: 153, with 1024 workgroups 171).
constexpr int kScanGrid = 256;

// Workgroups of four waves of the preparation, two a CU, which go on to further units
constexpr int kPrepareGrid = 512;

// Requests of at most this many tokens are taken token after token.  Both ways take
// as long between 21 and 36: 1, 8 and 32 requests of 64 heads of 128 x 128 17, 40 and
// 114 us at 16 tokens and 0.5, 1.9 and 5.2 a further one; in chunks 24, 46 and 135.
constexpr int kFewTokens = 20;

// Chunk slots of a call (first_slot), and bytes of a slot's records and decay
int64_t chunk_slots(const GdnCall& c) { return c.n_tokens / kChunk + c.n_requests; }
int64_t record_bytes(bool delta) {
  return delta ? Record<true>::kBytes : Record<false>::kBytes;
}

template <int DK, bool DELTA, int WAVES>
void launch_prepare(const GdnArgs& a, const GdnCall& c, int waves, hipStream_t stream) {
  const int units = static_cast<int>(chunk_slots(c) * c.n_k_heads);
  const int workgroups = WAVES == 4 && units > kPrepareGrid ? kPrepareGrid : units;
  prepare_kernel<DK, DELTA, WAVES>
      <<<static_cast<unsigned>(workgroups + (waves + WAVES - 1) / WAVES), WAVES * 64, 0, stream>>>(
          a, static_cast<int>(c.n_k_heads), units, workgroups);
}

template <int DK, bool DELTA>
void launch_dk(GdnArgs a, const GdnCall& c, hipStream_t stream) {
  const int waves = static_cast<int>(c.n_requests * c.n_heads * ((c.dv + 31) / 32));
  a.few = 0x7FFFFFFF;
  if (c.max_len <= kFewTokens) {
    // Few waves wait for their own operations: 16 columns each where 32 give at most
    // one wave to every other SIMD (16 tokens, 64 heads of 128 x 128: 21 us against 17,
    // 2 requests 22 and 17.6, 4 requests 24.6 and 27.4).
    if (waves <= 512) {
      const unsigned narrow = static_cast<unsigned>(c.n_requests * c.n_heads * (c.dv / 16));
      gdn_tokens_kernel<DK, DELTA, 4><<<(narrow + 3) / 4, 256, 0, stream>>>(a);
    } else {
      gdn_tokens_kernel<DK, DELTA, 8><<<static_cast<unsigned>((waves + 3) / 4), 256, 0, stream>>>(a);
    }
    return;
  }
  a.few = kFewTokens;
  a.records = static_cast<uint8_t*>(c.workspace);
  a.decays = reinterpret_cast<float*>(a.records + chunk_slots(c) * c.n_heads * record_bytes(DELTA));
  if (a.group == 1) launch_prepare<DK, DELTA, 1>(a, c, waves, stream);
  else if (a.group == 2) launch_prepare<DK, DELTA, 2>(a, c, waves, stream);
  else launch_prepare<DK, DELTA, 4>(a, c, waves, stream);
  const int items = a.group * static_cast<int>((c.dv + kScanCols - 1) / kScanCols);
  a.parts = static_cast<int>((7 + c.n_k_heads) / c.n_k_heads);
  while (items % a.parts != 0 && a.parts < 64) ++a.parts;
  if (items % a.parts != 0) a.parts = 1;
  a.share = items / a.parts;
  // a multiple of 8 that has every part of every key head
  const int64_t blocks = (c.n_requests * c.n_k_heads * a.parts + 7) / 8 * 8 * a.share;
  scan_kernel<DK, DELTA><<<static_cast<unsigned>(blocks < kScanGrid ? blocks : kScanGrid),
                           kScanThreads, 0, stream>>>(a);
}

}  // namespace

int64_t gdn_workspace(const GdnCall& c) {
  if (c.max_len <= kFewTokens) return 0;
  return chunk_slots(c) * c.n_heads * (record_bytes(c.beta != nullptr) + 4);
}

hipError_t launch_gdn(const GdnCall& c, hipStream_t stream) {
  if (c.n_tokens == 0) return hipSuccess;
  const GdnArgs a = args_of(c);
  if (c.dk == 64) c.beta ? launch_dk<64, true>(a, c, stream) : launch_dk<64, false>(a, c, stream);
  else c.beta ? launch_dk<128, true>(a, c, stream) : launch_dk<128, false>(a, c, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
