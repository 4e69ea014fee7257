// Attention of packed new tokens over a paged KV cache or over the packed
// prompt itself, for gfx950.
//
//   o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(c q.k_j - m),
//   c = scale log2 e,  m a running upper bound of c q.k_j,
//
// over the keys j that the row sees: j <= its position p (causal), j > p -
// window, j < kv length.  A row that sees none gives zeros.
//
// Rows.  The heads of one key/value head's group share its keys, so row R =
// token * group + head-in-group of a request is one query, and a workgroup
// takes a tile of consecutive rows of one request and key/value head: a
// decode token brings its whole group to each key, a chunk fills every row.
//
// Layout.  S^T = K Q^T, so that a query is a lane's column: the running
// maximum and sum stay in one register per lane and the weights of a lane
// are already the B operand of O^T = V^T P^T.  A lane's S^T registers hold
// keys 16 s + 8 e + 4 h + (0..3) (h the half-wave, e = 0, 1); the second
// product may take the 16 keys of a step in any order, so V^T is read in
// that one: two transposing LDS reads of 4 keys each per operand.
//
// Staging.  K and V go through registers into LDS (E4M3 codes are widened
// there once per workgroup and not once per wave: K to bf16, V to fp16, both
// exact), two tiles deep: while a tile is used the next one is in flight.
// 16-byte chunks of a row are exchanged by an exclusive or with the row
// number so that the fragment reads of 16 rows fall on different banks.
//
// Splits.  With few tiles the keys are cut into chunks that other
// workgroups take; each leaves its sums in binary32 with its bound, and
// combine_kernel joins them in chunk order (no atomics: results do not
// depend on timing).
//
// Precision.  Scores, bounds, sums and outputs are binary32.  The weights
// are rounded to the type of the second product: bf16 next to bf16 values,
// fp16 next to E4M3 ones.  That rounding is of the size of the bf16
// output's own.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "internal.h"
#include "kv_device.h"

namespace nvfp4 {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kTileRows = 128;         // rows of a workgroup, 32 a wave
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kNegInf = -__builtin_inff();

struct Args {
  const uint8_t* q;
  int64_t q_token, q_head;                        // bytes, here and below
  const uint8_t* k;
  const uint8_t* v;
  int64_t k_token, k_head, v_token, v_head, page_stride;
  uint8_t* out;
  int64_t out_token, out_head;
  const int32_t* table;
  int64_t ld_table;
  const int32_t* cu;
  const int32_t* kv_lens;
  const float* k_scale;
  const float* v_scale;
  float* part;                                    // [split][token * head][d]
  float* part_ml;                                 // [split][token * head][2]
  float scale_log2;
  int n_requests, n_tokens, n_heads, n_kv_heads, n_pages;
  FastDiv group, page;
  int64_t cols_len;                               // columns * page size
  int max_kv, causal, window, tiles, splits, chunk;
};

__device__ __forceinline__ int clampi(int64_t x, int64_t lo, int64_t hi) {
  return static_cast<int>(x < lo ? lo : x > hi ? hi : x);
}

// First tile of request i: floor(rows before / kTileRows) + i leaves every
// request at least the tiles it fills, without a prefix sum of its own.
__device__ __forceinline__ int64_t first_tile(const Args& a, int i) {
  const int64_t rows = static_cast<int64_t>(clampi(a.cu[i], 0, a.n_tokens)) * a.group.d;
  return rows / kTileRows + i;
}

// The request of tile t: the last i with first_tile(i) <= t (or, BY_TOKEN,
// with cu[i] <= t).  Each round the wave's 64 lanes probe 64 places.
template <bool BY_TOKEN>
__device__ __forceinline__ int find_request(const Args& a, int64_t t) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = a.n_requests;
  while (n > 1) {
    const int step = (n + 63) >> 6;
    const int at = lo + lane * step;
    const bool in = lane * step < n;
    const bool le = in && (BY_TOKEN ? static_cast<int64_t>(a.cu[at]) : first_tile(a, at)) <= t;
    const int c = __popcll(__ballot(le));
    const int skip = (c > 0 ? c - 1 : 0) * step;
    lo += skip;
    n = n - skip < step ? n - skip : step;
  }
  return lo;
}

// What a tile of rows of one request works on.
struct Span {
  int token0, n_new, kv;     // first token, tokens, keys of the request
  int row0;                  // first row of the tile within the request
  int lo, hi;                // keys that some row of the tile sees
  int start;                 // lo rounded down to whole 16-key groups
};

__device__ __forceinline__ void sees(const Args& a, const Span& s, int token, int* lo, int* hi) {
  const int64_t pos = static_cast<int64_t>(s.kv) - s.n_new + token;
  *hi = a.causal ? clampi(pos + 1, 0, s.kv) : s.kv;
  *lo = a.window ? clampi(pos - a.window + 1, 0, s.kv) : 0;
}

__device__ __forceinline__ Span span_of(const Args& a, int r, int row0, int rows) {
  Span s;
  s.token0 = clampi(a.cu[r], 0, a.n_tokens);
  s.n_new = clampi(a.cu[r + 1], s.token0, a.n_tokens) - s.token0;
  s.kv = a.kv_lens ? clampi(a.kv_lens[r], 0, a.cols_len < a.max_kv ? a.cols_len : a.max_kv)
                   : s.n_new;
  s.row0 = row0;
  s.lo = s.hi = 0;
  const int last_row = s.n_new * static_cast<int>(a.group.d) - 1;
  if (row0 <= last_row) {
    const int end = row0 + rows - 1;
    int unused;
    sees(a, s, static_cast<int>(a.group.div(row0)), &s.lo, &unused);
    sees(a, s, static_cast<int>(a.group.div(end < last_row ? end : last_row)), &unused, &s.hi);
  }
  s.start = s.lo & ~15;
  return s;
}

// Chunks that the keys of a tile are cut into.
__device__ __forceinline__ int splits_of(const Args& a, const Span& s) {
  const int n = (s.hi - s.start + a.chunk - 1) / a.chunk;
  return n < 1 ? 1 : n > a.splits ? a.splits : n;
}

// ---------------------------------------------------------------- staging

__device__ const u32x4 kZeros[64] = {};           // a row for pages out of range

template <int D, bool FP8>
struct Tile {
  static constexpr int kKeys = D > 128 ? 32 : 64;       // keys of a tile
  static constexpr int kRows = kKeys / 4;               // of a wave's share: within one page
  static constexpr int kChunks = D * (FP8 ? 1 : 2) / 16;    // 16-byte loads of a row
  static constexpr int kLoads = kRows * kChunks / 64;   // a lane's
  static constexpr int kBytes = kKeys * D * 2;          // in LDS
  // LDS bytes of 16-byte chunk c of row r.  K: the 16 rows that a fragment
  // read touches at once differ in their place; V: the 4 rows of a
  // transposing read do, by whole 64-byte pieces.
  static __device__ __forceinline__ int k_at(int r, int c) {
    return r * (D * 2) + ((c ^ (D == 64 ? (r >> 1) & 7 : r & 15)) << 4);
  }
  static __device__ __forceinline__ int v_at(int r, int c) {
    return r * (D * 2) + ((c ^ (D == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2)) << 4);
  }
};

// 4 codes of one dword to 4 values, K as bf16 and V as fp16 (both exact).
template <bool IS_V>
__device__ __forceinline__ u32x2 widen4(unsigned w) {
  u32x2 r;
  if constexpr (IS_V) {
    r[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false));
    r[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true));
  } else {
    r[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
    r[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true));
  }
  return r;
}

template <int D, bool FP8>
struct Stage {
  using T = Tile<D, FP8>;
  u32x4 k[T::kLoads], v[T::kLoads];

  // Keys [key0, key0 + kKeys) of the request: this wave's rows.  Rows
  // outside [lo, hi) are read at the nearest one inside, so that whatever
  // a cache holds past a request's end is never used; pages out of range
  // read as zeros.
  __device__ __forceinline__ void load(const Args& a, const Span& s, const int32_t* row_of_table,
                                       int64_t head_k, int64_t head_v, int key0, int wave) {
    const int lane = threadIdx.x & 63;
    int g = key0 + wave * T::kRows;               // uniform; 16 keys share a page
    const int last = (s.hi - 1) & ~(T::kRows - 1);
    g = g < last ? g : last;
    const uint8_t* kb;
    const uint8_t* vb;
    int64_t kt = a.k_token, vt = a.v_token;
    if (row_of_table) {
      const int blk = static_cast<int>(a.page.div(static_cast<unsigned>(g)));
      const int id = row_of_table[blk];
      const int off = g - blk * static_cast<int>(a.page.d);
      if (id >= 0 && id < a.n_pages) {
        kb = a.k + id * a.page_stride + head_k + off * kt;
        vb = a.v + id * a.page_stride + head_v + off * vt;
      } else {
        kb = vb = reinterpret_cast<const uint8_t*>(kZeros);
        kt = vt = 0;
      }
    } else {
      kb = a.k + (static_cast<int64_t>(s.token0) + g) * kt + head_k;
      vb = a.v + (static_cast<int64_t>(s.token0) + g) * vt + head_v;
    }
    const int first = s.lo - g, end = s.hi - 1 - g;
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) {
      const int at = i * 64 + lane;
      int r = at / T::kChunks;
      const int c = at % T::kChunks;
      r = r < first ? first : r;
      r = r > end ? end : r;
      k[i] = *reinterpret_cast<const u32x4*>(kb + r * static_cast<int>(kt) + c * 16);
      v[i] = *reinterpret_cast<const u32x4*>(vb + r * static_cast<int>(vt) + c * 16);
    }
  }

  __device__ __forceinline__ void store(uint8_t* lds_k, uint8_t* lds_v, int wave) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i) {
      const int at = i * 64 + lane;
      const int r = wave * T::kRows + at / T::kChunks, c = at % T::kChunks;
      if constexpr (FP8) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const u32x2 k0 = widen4<false>(k[i][2 * p]), k1 = widen4<false>(k[i][2 * p + 1]);
          const u32x2 v0 = widen4<true>(v[i][2 * p]), v1 = widen4<true>(v[i][2 * p + 1]);
          *reinterpret_cast<u32x4*>(lds_k + T::k_at(r, 2 * c + p)) = u32x4{k0[0], k0[1], k1[0], k1[1]};
          *reinterpret_cast<u32x4*>(lds_v + T::v_at(r, 2 * c + p)) = u32x4{v0[0], v0[1], v1[0], v1[1]};
        }
      } else {
        *reinterpret_cast<u32x4*>(lds_k + T::k_at(r, c)) = k[i];
        *reinterpret_cast<u32x4*>(lds_v + T::v_at(r, c)) = v[i];
      }
    }
  }
};

// Barrier for LDS alone: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

__device__ __forceinline__ s16x4 read_tr(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)(p));
}

// max of a value over the two half-waves that share a column.
__device__ __forceinline__ float half_max(float x) {
  const unsigned u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const unsigned u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <bool HALF>
__device__ __forceinline__ unsigned pack2(float x, float y) {
  const f32x2 p = {x, y};
  if constexpr (HALF) return __builtin_bit_cast(unsigned, __builtin_convertvector(p, half2_t));
  else return __builtin_bit_cast(unsigned, __builtin_convertvector(p, bf16x2));
}

// ---------------------------------------------------------------- kernel

// One tile of 128 rows; 4 waves, 32 rows each.
template <int D, bool FP8>
__global__ void __launch_bounds__(256, D > 128 ? 1 : 2) attn_tile_kernel(Args a) {
  using T = Tile<D, FP8>;
  constexpr int kSteps = D / 16;          // of the first product
  constexpr int kBlocks = T::kKeys / 32;  // key blocks of a tile
  constexpr int kDb = D / 32;             // d blocks of the output
  // weights are at most 2^kSlack: the bound is moved only when a score
  // passes it by more (fp16 weights are kept 2^6 higher, away from its
  // subnormals; 2^14 is still in range)
  constexpr float kSlack = 8.0f;
  constexpr float kLift = FP8 ? 6.0f : 0.0f;
  __shared__ __attribute__((aligned(16))) uint8_t lds[4 * T::kBytes];

  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int kvh = blockIdx.x % a.n_kv_heads;
  const int rest = blockIdx.x / a.n_kv_heads;
  const int split = rest % a.splits;
  const int tile = a.tiles - 1 - rest / a.splits;    // the longest rows of a prompt first

  const int r = __builtin_amdgcn_readfirstlane(find_request<false>(a, tile));
  const int64_t row0 = (tile - first_tile(a, r)) * kTileRows;
  const int group = static_cast<int>(a.group.d);
  const int64_t n_rows = static_cast<int64_t>(clampi(a.cu[r + 1], 0, a.n_tokens) -
                                              clampi(a.cu[r], 0, a.n_tokens)) * group;
  if (row0 < 0 || row0 >= n_rows) return;
  const Span s = span_of(a, r, static_cast<int>(row0), kTileRows);
  const int splits = splits_of(a, s);
  if (split >= splits) return;
  const int begin = s.start + split * a.chunk;
  const int end = split == splits - 1 ? s.hi : begin + a.chunk;

  // this lane's row
  const int row = s.row0 + wave * 32 + col;
  const bool real = row < n_rows;
  const int token = static_cast<int>(a.group.div(real ? row : 0));
  const int head = kvh * group + (real ? row - token * group : 0);
  int see_lo = 0, see_hi = 0;
  if (real) sees(a, s, token, &see_lo, &see_hi);
  // what all rows of the wave see, for tiles that need no mask
  int all_lo = see_lo, all_hi = see_hi, any_lo = real ? see_lo : 0x7FFFFFFF, any_hi = see_hi;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    all_lo = max(all_lo, __shfl_xor(all_lo, off));
    all_hi = min(all_hi, __shfl_xor(all_hi, off));
    any_lo = min(any_lo, __shfl_xor(any_lo, off));
    any_hi = max(any_hi, __shfl_xor(any_hi, off));
  }
  all_lo = __builtin_amdgcn_readfirstlane(all_lo);
  all_hi = __builtin_amdgcn_readfirstlane(all_hi);
  any_lo = __builtin_amdgcn_readfirstlane(any_lo);
  any_hi = __builtin_amdgcn_readfirstlane(any_hi);

  bf16x8 qf[kSteps];
  {
    const uint8_t* qp = a.q + (static_cast<int64_t>(s.token0) + token) * a.q_token + head * a.q_head;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      qf[i] = *reinterpret_cast<const bf16x8*>(qp + i * 32 + half * 16);
  }
  // a scale of zero makes every score 0; it must not make -inf * 0 of a
  // masked one
  const float c = FP8 ? fmaxf(a.scale_log2 * *a.k_scale, 0x1p-120f) : a.scale_log2;

  f32x16 acc[kDb];
#pragma unroll
  for (int b = 0; b < kDb; ++b)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[b][i] = 0.0f;
  float m = kNegInf, l = 0.0f;

  const int32_t* table = a.table ? a.table + r * a.ld_table : nullptr;
  const int64_t head_k = kvh * a.k_head, head_v = kvh * a.v_head;
  Stage<D, FP8> st;
  if (begin < end) st.load(a, s, table, head_k, head_v, begin, wave);
  int buf = 0;
  for (int key0 = begin; key0 < end; key0 += T::kKeys, buf ^= 1) {
    uint8_t* lk = lds + buf * 2 * T::kBytes;
    uint8_t* lv = lk + T::kBytes;
    // the waves still at the tile before last have passed the last barrier
    st.store(lk, lv, wave);
    if (key0 + T::kKeys < end) st.load(a, s, table, head_k, head_v, key0 + T::kKeys, wave);
    lds_barrier();
    if (key0 >= any_hi || key0 + T::kKeys <= any_lo) continue;    // no row sees the tile

    f32x16 sc[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[b][i] = 0.0f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const bf16x8 kf = *reinterpret_cast<const bf16x8*>(lk + T::k_at(32 * b + col, 2 * i + half));
        sc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[i], sc[b], 0, 0, 0);
      }
    }
    if (key0 < all_lo || key0 + T::kKeys > all_hi) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = key0 + 32 * b + 8 * (i >> 2) + 4 * half + (i & 3);
          if (j < see_lo || j >= see_hi) sc[b][i] = kNegInf;
        }
    }
    float top = sc[0][0];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[b][i]);
    top = half_max(top) * c;
    if (__any(top > m + kSlack)) {
      const float m2 = fmaxf(m, top);
      const float f = m2 == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - m2);
      m = m2;
      l *= f;
#pragma unroll
      for (int b = 0; b < kDb; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[b][i] *= f;
    }
    const float shift = (m == kNegInf ? 0.0f : m) - kLift;
    unsigned pw[kBlocks][8];
    float sum = 0.0f;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[b][i], c, -shift));
        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[b][i + 1], c, -shift));
        sum += p0 + p1;
        pw[b][i >> 1] = pack2<FP8>(p0, p1);
      }
    l += sum;
    // O^T += V^T P^T, 16 keys a step
#pragma unroll
    for (int t = 0; t < T::kKeys / 16; ++t) {
      const u32x4 pf = {pw[t >> 1][4 * (t & 1)], pw[t >> 1][4 * (t & 1) + 1],
                        pw[t >> 1][4 * (t & 1) + 2], pw[t >> 1][4 * (t & 1) + 3]};
      const int vr = 16 * t + 4 * half + ((lane & 15) >> 2);
#pragma unroll
      for (int b = 0; b < kDb; ++b) {
        const int vc = 4 * b + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
        const s16x4 v0 = read_tr(lv + T::v_at(vr, vc) + 8 * (lane & 1));
        const s16x4 v1 = read_tr(lv + T::v_at(vr + 8, vc) + 8 * (lane & 1));
        const s16x8 vf = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
        if constexpr (FP8)
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, vf),
                                                          __builtin_bit_cast(half8_t, pf), acc[b], 0, 0, 0);
        else
          acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vf),
                                                           __builtin_bit_cast(bf16x8, pf), acc[b], 0, 0, 0);
      }
    }
  }
  l = half_sum(l);
  if (!real) return;
  const int64_t out_row = static_cast<int64_t>(s.token0) + token;
  if (splits == 1) {
    const float inv = l > 0.0f ? (FP8 ? *a.v_scale : 1.0f) / l : 0.0f;
    uint8_t* op = a.out + out_row * a.out_token + head * a.out_head;
#pragma unroll
    for (int b = 0; b < kDb; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x2 w = {pack2<false>(acc[b][4 * i] * inv, acc[b][4 * i + 1] * inv),
                         pack2<false>(acc[b][4 * i + 2] * inv, acc[b][4 * i + 3] * inv)};
        *reinterpret_cast<u32x2*>(op + (32 * b + 8 * i + 4 * half) * 2) = w;
      }
  } else {
    const int64_t at = (static_cast<int64_t>(split) * a.n_tokens + out_row) * a.n_heads + head;
    float* pp = a.part + at * D;
#pragma unroll
    for (int b = 0; b < kDb; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<f32x4*>(pp + 32 * b + 8 * i + 4 * half) =
            f32x4{acc[b][4 * i], acc[b][4 * i + 1], acc[b][4 * i + 2], acc[b][4 * i + 3]};
    if (half == 0) *reinterpret_cast<f32x2*>(a.part_ml + at * 2) = f32x2{m, l};
  }
}

// Joins the chunks of each row: one wave a row.
template <int D, bool FP8>
__global__ void __launch_bounds__(256) combine_kernel(Args a) {
  constexpr int kEach = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (row >= static_cast<int64_t>(a.n_tokens) * a.n_heads) return;
  const int t = static_cast<int>(row / a.n_heads), head = static_cast<int>(row % a.n_heads);
  const int r = find_request<true>(a, t);
  const int group = static_cast<int>(a.group.d);
  const int token0 = clampi(a.cu[r], 0, a.n_tokens);
  if (t >= a.cu[r + 1] || t < token0) return;        // rows of no request
  const int tile_row = ((t - token0) * group + head % group) / kTileRows * kTileRows;
  const Span s = span_of(a, r, tile_row, kTileRows);
  const int splits = splits_of(a, s);
  if (splits == 1) return;
  const int64_t rows = static_cast<int64_t>(a.n_tokens) * a.n_heads;
  float m = kNegInf;
  for (int i = 0; i < splits; ++i) {
    const f32x2 ml = *reinterpret_cast<const f32x2*>(a.part_ml + (i * rows + row) * 2);
    if (ml[1] > 0.0f) m = fmaxf(m, ml[0]);
  }
  float l = 0.0f, o[kEach] = {};
  for (int i = 0; i < splits; ++i) {
    const f32x2 ml = *reinterpret_cast<const f32x2*>(a.part_ml + (i * rows + row) * 2);
    const float f = ml[1] > 0.0f ? __builtin_amdgcn_exp2f(ml[0] - m) : 0.0f;
    l = __builtin_fmaf(ml[1], f, l);
    const float* p = a.part + (i * rows + row) * D + lane * kEach;
#pragma unroll
    for (int e = 0; e < kEach; ++e) o[e] = __builtin_fmaf(p[e], f, o[e]);
  }
  const float inv = l > 0.0f ? (FP8 ? *a.v_scale : 1.0f) / l : 0.0f;
  __bf16* op = reinterpret_cast<__bf16*>(a.out + t * a.out_token + head * a.out_head) + lane * kEach;
#pragma unroll
  for (int e = 0; e < kEach; ++e) op[e] = static_cast<__bf16>(o[e] * inv);
}

// ------------------------------------------------------------------ host

constexpr int64_t kCus = 256;

struct Plan {
  int64_t tiles, splits, chunk;
};

Plan plan_of(const AttnCall& c) {
  Plan p;
  const int64_t group = c.n_heads / c.n_kv_heads;
  p.tiles = c.n_tokens * group / kTileRows + c.n_requests;
  // keys of the longest tile, its first group rounded down included
  int64_t keys = c.table ? c.max_kv : c.max_new;
  const int64_t tokens = kTileRows / group + 2;
  if (c.window && keys > c.window + tokens) keys = c.window + tokens;
  keys += 15;
  const int64_t wgs = p.tiles * c.n_kv_heads;
  // fill the CUs twice over, with chunks of at least 256 keys
  int64_t want = (2 * kCus + wgs - 1) / wgs;
  const int64_t most = (keys + 255) / 256;
  want = want < most ? want : most;
  p.chunk = ((keys + want - 1) / want + 127) / 128 * 128;
  p.splits = (keys + p.chunk - 1) / p.chunk;
  return p;
}

template <int D, bool FP8>
void launch(const Args& a, hipStream_t stream) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(a.tiles) * a.splits * a.n_kv_heads);
  attn_tile_kernel<D, FP8><<<grid, 256, 0, stream>>>(a);
  if (a.splits > 1) {
    const int64_t rows = static_cast<int64_t>(a.n_tokens) * a.n_heads;
    combine_kernel<D, FP8><<<static_cast<unsigned>((rows + 3) / 4), 256, 0, stream>>>(a);
  }
}

}  // namespace

int64_t attention_workspace(const AttnCall& c) {
  const Plan p = plan_of(c);
  if (p.splits <= 1) return 0;
  return p.splits * c.n_tokens * c.n_heads * (c.d + 2) * 4;
}

hipError_t launch_attention(const AttnCall& c, hipStream_t stream) {
  const Plan p = plan_of(c);
  const bool paged = c.table != nullptr;
  const int64_t cs = paged && c.pool.fp8 ? 1 : 2;
  Args a;
  a.q = static_cast<const uint8_t*>(c.q.p);
  a.q_token = c.q.token * 2;
  a.q_head = c.q.head * 2;
  a.k = static_cast<const uint8_t*>(paged ? c.pool.k : c.k.p);
  a.v = static_cast<const uint8_t*>(paged ? c.pool.v : c.v.p);
  a.k_token = (paged ? c.pool.token_stride : c.k.token) * cs;
  a.k_head = (paged ? c.pool.head_stride : c.k.head) * cs;
  a.v_token = (paged ? c.pool.token_stride : c.v.token) * cs;
  a.v_head = (paged ? c.pool.head_stride : c.v.head) * cs;
  a.page_stride = paged ? c.pool.page_stride * cs : 0;
  a.out = static_cast<uint8_t*>(c.out);
  a.out_token = c.out_token * 2;
  a.out_head = c.out_head * 2;
  a.table = c.table;
  a.ld_table = c.ld_table;
  a.cu = c.cu;
  a.kv_lens = c.kv_lens;
  a.k_scale = c.pool.k_scale;
  a.v_scale = c.pool.v_scale;
  a.part = static_cast<float*>(c.workspace);
  a.part_ml = a.part + p.splits * c.n_tokens * c.n_heads * c.d;
  a.scale_log2 = c.scale * kLog2e;
  a.n_requests = static_cast<int>(c.n_requests);
  a.n_tokens = static_cast<int>(c.n_tokens);
  a.n_heads = static_cast<int>(c.n_heads);
  a.n_kv_heads = static_cast<int>(c.n_kv_heads);
  a.n_pages = paged ? static_cast<int>(c.pool.n_pages) : 0;
  a.group = FastDiv::of(static_cast<unsigned>(c.n_heads / c.n_kv_heads));
  a.page = FastDiv::of(paged ? static_cast<unsigned>(c.pool.page_size) : 16u);
  a.cols_len = paged ? c.cols * c.pool.page_size : 0;
  a.max_kv = static_cast<int>(c.max_kv);
  a.causal = c.causal;
  a.window = static_cast<int>(c.window);
  a.tiles = static_cast<int>(p.tiles);
  a.splits = static_cast<int>(p.splits);
  a.chunk = static_cast<int>(p.chunk);
  const bool fp8 = paged && c.pool.fp8;
  if (c.d == 64) fp8 ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
  else if (c.d == 128) fp8 ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
  else fp8 ? launch<256, true>(a, stream) : launch<256, false>(a, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
