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
// Staging of tiles.  Two tiles of K and V in LDS: while one is used the next
// is in flight, bf16 from memory straight to LDS, E4M3 codes through
// registers, where they are widened once per workgroup and not once per wave
// (K to bf16, V to fp16, both exact).  16-byte chunks of a row are exchanged
// by an exclusive or with the row number so that the operand reads of 16 rows
// fall on different banks (no conflict counted).
//
// Requests of few rows (decodes) have no use for tiles: they are bound by the
// read of their keys and values, which a kernel of its own streams.
//
// Chunks.  With few tiles, and for decodes, the keys are cut into chunks that
// other workgroups take; each leaves its sums in binary32 with its bound, and
// combine_kernel joins them in a fixed order (no atomics: results do not
// depend on timing).
//
// Precision.  Scores, bounds, sums and outputs are binary32.  The weights
// are rounded to the type of the second product: bf16 next to bf16 values,
// fp16 next to E4M3 ones.  That rounding is of the size of the bf16
// output's own.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "kv_cut.h"
#include "kv_device.h"
#include "kv_place.h"

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
constexpr int kFewRows = 16;           // most rows of a request that few_rows takes
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
  // sums of chunks of keys, [slot][d] and [slot][2] (bound, sum of weights)
  float* part;
  float* part_ml;
  float scale_log2;
  int n_requests, n_tokens, n_heads, n_kv_heads, n_pages;
  FastDiv group, page;
  int64_t cols_len;                               // columns * page size
  int max_kv, causal, window, tiles;
  int tile_blocks;                                // workgroups of the tiles
  int splits, chunk;                              // chunks of the tiles' keys
  // requests of few rows (few_pieces: 0, none): most rows of one (and places
  // of a piece's sums), most pieces that their keys are cut into; keys of a
  // piece and pieces of a request, or 0 for a cut that the kernel makes from
  // the lengths; workgroups
  int few_rows, few_pieces, few_chunk, few_splits, few_blocks;
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

// Chunks that the keys of a span are cut into.
__device__ __forceinline__ int splits_of(const Span& s, int chunk, int most) {
  return chunks_of(s.hi - s.start, chunk, most);
}

// Places of a chunk's sums: of a row of a tile, of a row of a few-row request.
__device__ __forceinline__ int64_t tile_slot(const Args& a, int split, int64_t token, int head) {
  return (static_cast<int64_t>(split) * a.n_tokens + token) * a.n_heads + head;
}
__device__ __forceinline__ int64_t few_slot(const Args& a, int piece, int kvh, int row) {
  const int64_t before = a.splits > 1 ? tile_slot(a, a.splits, 0, 0) : 0;
  return before + (static_cast<int64_t>(piece) * a.n_kv_heads + kvh) * a.few_rows + row;
}

// How the keys of the requests of few rows are cut into pieces of equal
// length (kv_cut.h), a request's pieces one after another.  Up to kPlanned
// requests the cut follows the lengths (a pass over them, 64 at a time, by
// every wave): 32 requests of 32768 E4M3 keys of 4 heads of 256 take 325 us,
// with 2048 keys a piece 353 us; 64 requests of 1 to 16384 keys 77 us, with
// 2048 keys a piece 92 us, 1024 80 us, 4096 116 us.
constexpr int kPlanned = 256;
// Fewest keys of a piece.  A small call is bound by its launches, so the choice
// shows little: d 64, 256 or 512 keys: within 1 us from 1 to 256 requests
// (1024: 43 instead of 36 us for 64 ragged ones of up to 4000); d 256, 256 or 512
// keys: 19 and 21 us for 8 requests of 2000 keys, 26 and 23 us for 32 of 1000.
constexpr int few_least(int d) { return d == 64 ? 256 : 512; }
struct Cut {
  int chunk, pieces;
  int first[kPlanned / 64];        // lane i: first piece of requests i, 64 + i, ...
};

// Inclusive sums over the lanes of non-negative values, in registers (DPP: a
// shift of 1, 2, 4, 8 in each row of 16 lanes, then the rows' ends passed on).
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_zero(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int lane_sums(int x) {
  x += dpp_or_zero<0x111, 0xF>(x);
  x += dpp_or_zero<0x112, 0xF>(x);
  x += dpp_or_zero<0x114, 0xF>(x);
  x += dpp_or_zero<0x118, 0xF>(x);
  x += dpp_or_zero<0x142, 0xA>(x);
  x += dpp_or_zero<0x143, 0xC>(x);
  return x;
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_or_zero(float x) {
  return __uint_as_float(dpp_or_zero<CTRL, ROWS>(static_cast<int>(__float_as_uint(x))));
}
// Sum and maximum over the wave of non-negative values (in lane 63's order:
// the same in every wave).
__device__ __forceinline__ float of_last(float x) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), 63));
}
__device__ __forceinline__ float wave_sum(float x) {
  x += dpp_or_zero<0x111, 0xF>(x);
  x += dpp_or_zero<0x112, 0xF>(x);
  x += dpp_or_zero<0x114, 0xF>(x);
  x += dpp_or_zero<0x118, 0xF>(x);
  x += dpp_or_zero<0x142, 0xA>(x);
  x += dpp_or_zero<0x143, 0xC>(x);
  return of_last(x);
}
__device__ __forceinline__ float wave_max(float x) {
  x = fmaxf(x, dpp_or_zero<0x111, 0xF>(x));
  x = fmaxf(x, dpp_or_zero<0x112, 0xF>(x));
  x = fmaxf(x, dpp_or_zero<0x114, 0xF>(x));
  x = fmaxf(x, dpp_or_zero<0x118, 0xF>(x));
  x = fmaxf(x, dpp_or_zero<0x142, 0xA>(x));
  x = fmaxf(x, dpp_or_zero<0x143, 0xC>(x));
  return of_last(x);
}

template <int D>
__device__ __forceinline__ Cut cut_of(const Args& a) {
  Cut c = {a.few_chunk, a.few_pieces, {}};
  if (a.few_chunk) return c;
  const int lane = threadIdx.x & 63;
  int keys[kPlanned / 64];         // -1: not a request of few rows
  float total = 0.0f, most = 0.0f, n = 0.0f;
#pragma unroll
  for (int q = 0; q < kPlanned / 64; ++q) {
    keys[q] = -1;
    if (q * 64 >= a.n_requests) continue;
    const int i = q * 64 + lane;
    if (i < a.n_requests) {
      const Span s = span_of(a, i, 0, kFewRows);
      const int64_t rows = static_cast<int64_t>(s.n_new) * a.group.d;
      if (rows > 0 && rows <= a.few_rows) {
        keys[q] = s.hi - s.start;
        total += static_cast<float>(keys[q]);
        most = fmaxf(most, static_cast<float>(keys[q]));
        n += 1.0f;
      }
    }
  }
  total = wave_sum(total);
  most = wave_max(most);
  n = wave_sum(n);
  c.chunk = __builtin_amdgcn_readfirstlane(piece_keys(total, most, n, a.n_kv_heads, few_least(D)));
  const float per_key = 1.0f / static_cast<float>(c.chunk);
  int before = 0;
#pragma unroll
  for (int q = 0; q < kPlanned / 64; ++q) {
    c.first[q] = before;
    if (q * 64 >= a.n_requests) continue;
    const int count = keys[q] < 0 ? 0 : pieces_of(keys[q], c.chunk, per_key);
    const int sums = lane_sums(count);
    c.first[q] = before + sums - count;
    before += __builtin_amdgcn_readlane(sums, 63);
  }
  c.pieces = before;
  return c;
}

// First piece of request r, and the request of a piece.
__device__ __forceinline__ int first_piece(const Args& a, const Cut& c, int r) {
  if (a.few_chunk) return r * a.few_splits;
  int f = 0;
#pragma unroll
  for (int q = 0; q < kPlanned / 64; ++q)
    if (r >> 6 == q) f = __builtin_amdgcn_readlane(c.first[q], r & 63);
  return f;
}
__device__ __forceinline__ int request_of(const Args& a, const Cut& c, int piece) {
  if (a.few_chunk) return piece / a.few_splits;
  int n = 0;                       // requests that begin at or before the piece
#pragma unroll
  for (int q = 0; q < kPlanned / 64; ++q)
    n += __popcll(__ballot(q * 64 + static_cast<int>(threadIdx.x & 63) < a.n_requests &&
                           c.first[q] <= piece));
  return n - 1;
}

// Tile `index` of the launch: its request and which of the request's tiles it
// is.  Up to kPlanned requests the tiles come by their place in the request,
// the last ones first: under a causal mask those have the most keys, and a
// long tile that starts late would end alone (7 prompts of up to 2001 tokens,
// d 256: 102 us in the requests' order, 99 us in this one; 3 chunks and 21
// decodes: 82 and 79 us; 16 requests of 5 tokens over 8192 keys: the same).
// With S(p) = sum_r max(0, tiles_r - p) tiles at places >= p, tile `index` is
// at the largest p with S(p) > index.
__device__ __forceinline__ int64_t rows_of(const Args& a, int r) {
  const int t0 = clampi(a.cu[r], 0, a.n_tokens);
  return static_cast<int64_t>(clampi(a.cu[r + 1], t0, a.n_tokens) - t0) * a.group.d;
}
__device__ __forceinline__ bool tile_of(const Args& a, int index, int* r, int* level) {
  if (a.n_requests > kPlanned) {
    const int tile = a.tiles - 1 - index;
    *r = __builtin_amdgcn_readfirstlane(find_request<false>(a, tile));
    // tiles before the first request's, where the offsets do not begin at 0
    *level = static_cast<int>(tile - first_tile(a, *r));
    return *level >= 0;
  }
  constexpr int kQ = kPlanned / 64;
  const int lane = threadIdx.x & 63;
  int tiles[kQ], most = 0, total = 0;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    tiles[q] = 0;
    if (q * 64 >= a.n_requests) continue;
    if (q * 64 + lane < a.n_requests) {
      const int64_t rows = rows_of(a, q * 64 + lane);
      if (!(a.few_pieces > 0 && rows <= a.few_rows))
        tiles[q] = static_cast<int>((rows + kTileRows - 1) / kTileRows);
    }
    most = max(most, tiles[q]);
    total += tiles[q];
  }
  most = static_cast<int>(wave_max(static_cast<float>(most)));
  if (index >= __builtin_amdgcn_readlane(lane_sums(total), 63)) return false;
  int lo = 0, hi = most, above = 0;     // S(lo) > index >= S(hi) = above
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    int n = 0;
#pragma unroll
    for (int q = 0; q < kQ; ++q) n += max(tiles[q] - mid, 0);
    n = __builtin_amdgcn_readlane(lane_sums(n), 63);
    if (n > index) {
      lo = mid;
    } else {
      hi = mid;
      above = n;
    }
  }
  int nth = index - above;              // among the requests with a tile at lo
  *level = lo;
  *r = 0;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const uint64_t have = __ballot(tiles[q] > lo);
    const int n = __popcll(have);
    if (nth >= 0 && nth < n) {
      const int before = __builtin_amdgcn_mbcnt_hi(static_cast<unsigned>(have >> 32),
                                                   __builtin_amdgcn_mbcnt_lo(static_cast<unsigned>(have), 0));
      const uint64_t it = __ballot(tiles[q] > lo && before == nth);
      *r = q * 64 + __builtin_ctzll(it);
    }
    nth -= n;
  }
  return true;
}

// ---------------------------------------------------------------- staging

// 16 bytes from global memory: said so, since a load that might be of LDS
// counts with the LDS reads and makes each of their waits wait for it.
// ONCE: nothing reads them again, so they need not displace what is cached.
template <bool ONCE>
__device__ __forceinline__ u32x4 load16b(const uint8_t* base, unsigned off) {
  typedef const __attribute__((address_space(1))) uint8_t* gptr;
  typedef const __attribute__((address_space(1))) u32x4* gvec;
  const gvec p = (gvec)((gptr)base + off);
  return ONCE ? __builtin_nontemporal_load(p) : *p;
}

__device__ const u32x4 kZeros[64] = {};           // a row for pages out of range

// A resource over the bytes from base on (32-bit offsets), and 16 bytes per
// lane from it straight to LDS at lds + 16 * lane.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const uint8_t* base) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  const unsigned lo = __builtin_amdgcn_readfirstlane(static_cast<unsigned>(p));
  const unsigned hi = __builtin_amdgcn_readfirstlane(static_cast<unsigned>(p >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(
      reinterpret_cast<void*>((static_cast<uint64_t>(hi) << 32) | lo), 0, 0x7FFFFFFF, 0x00020000);
}
__device__ __forceinline__ void lds_load16(__amdgpu_buffer_rsrc_t rsrc, uint8_t* lds, unsigned off) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)lds, 16,
                                           off, 0, 0, 0);
#endif
}

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
  static __device__ __forceinline__ int k_swap(int r) { return D == 64 ? (r >> 1) & 7 : r & 15; }
  static __device__ __forceinline__ int v_swap(int r) {
    return D == 64 ? ((r >> 1) & 1) << 2 : (r & 3) << 2;
  }
  static __device__ __forceinline__ int k_at(int r, int c) {
    return r * (D * 2) + ((c ^ k_swap(r)) << 4);
  }
  static __device__ __forceinline__ int v_at(int r, int c) {
    return r * (D * 2) + ((c ^ v_swap(r)) << 4);
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

// Page of a 16-key group: a scalar load, whatever the stores around it (the
// table does not change during a launch).
__device__ __forceinline__ int page_of(const Args& a, const int32_t* row_of_table, int key) {
  typedef const __attribute__((address_space(4))) int32_t* cptr;
  return ((cptr)row_of_table)[a.page.div(static_cast<unsigned>(key))];
}

// Where the ROWS keys from `key` on (of one 16-key group) are, and which of
// them may be read: rows outside [lo, hi) are read at the nearest one inside,
// so that whatever a cache holds past a request's end is never used.  A page
// out of range reads as zeros.
struct Place {
  const uint8_t* k;
  const uint8_t* v;
  RowBounds rows;
};
template <int ROWS>
__device__ __forceinline__ Place place_of(const Args& a, const Span& s, int64_t head_k,
                                          int64_t head_v, int key, int id) {
  const int g = group_at<ROWS>(s.hi, key);
  Place p = {a.k + head_k, a.v + head_v, rows_seen(s.lo, s.hi, g)};
  if (a.table) {
    const int off = g - static_cast<int>(a.page.div(static_cast<unsigned>(g)) * a.page.d);
    if (id >= 0 && id < a.n_pages) {
      const int64_t at = id * a.page_stride + off * a.k_token;    // K and V alike
      p.k += at;
      p.v += at;
    } else {
      p.k = p.v = reinterpret_cast<const uint8_t*>(kZeros);
      p.rows = {0, 0};                   // every row at the one of zeros
    }
  } else {
    p.k += (static_cast<int64_t>(s.token0) + g) * a.k_token;
    p.v += (static_cast<int64_t>(s.token0) + g) * a.v_token;
  }
  return p;
}

// A wave's rows of K or V of one tile on their way to LDS: bf16 straight
// from memory (no registers), E4M3 codes through registers, widened there.
template <int D, bool FP8, bool IS_V>
struct Stage {
  using T = Tile<D, FP8>;
  u32x4 x[FP8 ? T::kLoads : 1];

  __device__ __forceinline__ void load(const Place& p, int stride, int wave, uint8_t* lds) {
    const int lane = threadIdx.x & 63;
    const uint8_t* base = IS_V ? p.v : p.k;
    const int r0 = lane / T::kChunks, c0 = lane % T::kChunks;
    constexpr int kStep = 64 / T::kChunks;        // rows from one load to the next
    const ByteBounds bytes = bytes_seen(p.rows, stride);
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < T::kLoads; ++i)
        x[i] = load16b<false>(base, byte_of(r0 * stride + i * kStep * stride, bytes) + c0 * 16);
    } else {
      // LDS takes consecutive lanes' pieces one after another; which chunk of
      // the row a lane brings makes the exchange
      const auto rsrc = resource(base);
#pragma unroll
      for (int i = 0; i < T::kLoads; ++i) {
        const int r = wave * T::kRows % 16 + r0 + i * kStep;
        const int c = c0 ^ (IS_V ? T::v_swap(r) : T::k_swap(r));
        lds_load16(rsrc, lds + (wave * T::kLoads + i) * 1024,
                   byte_of(r0 * stride + i * kStep * stride, bytes) + c * 16);
      }
    }
  }

  // E4M3: the widened values to LDS.
  __device__ __forceinline__ void store(uint8_t* lds, int wave) const {
    if constexpr (FP8) {
      const int lane = threadIdx.x & 63;
#pragma unroll
      for (int i = 0; i < T::kLoads; ++i) {
        const int at = i * 64 + lane;
        const int r = wave * T::kRows + at / T::kChunks, c = at % T::kChunks;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const u32x2 w0 = widen4<IS_V>(x[i][2 * p]), w1 = widen4<IS_V>(x[i][2 * p + 1]);
          *reinterpret_cast<u32x4*>(lds + (IS_V ? T::v_at(r, 2 * c + p) : T::k_at(r, 2 * c + p))) =
              u32x4{w0[0], w0[1], w1[0], w1[1]};
        }
      }
    }
  }
};

// Every wave's part of the next tile is in LDS (loads to LDS count as vector
// memory) and its reads of this one are done.
__device__ __forceinline__ void tile_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);      // vmcnt(0) lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
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

// N instructions of a kind (0x008 MFMA, 0x100 LDS reads) next, in the order of
// these calls.
template <int KIND, int N>
__device__ __forceinline__ void order() {
  __builtin_amdgcn_sched_group_barrier(KIND, N, 0);
}

// The weights are 2^(c s - m) with a bound m that may be up to kSlack below
// the largest score: it is moved, and the sums with it, only when a score
// passes it by more.  fp16 weights (next to E4M3 values) are lifted away from
// fp16's subnormals, 2^(c s - m + kLift); 2^14 is still in its range.
constexpr float kSlack = 8.0f;
constexpr float kLift = 6.0f;
template <bool FP8>
__device__ __forceinline__ float shift_of(float m) {
  return (m == kNegInf ? 0.0f : m) - (FP8 ? kLift : 0.0f);
}
// Raises m to top; returns the factor of the sums so far.
__device__ __forceinline__ float moved(float* m, float top) {
  const float m2 = fmaxf(*m, top);
  const float f = m2 == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(*m - m2);
  *m = m2;
  return f;
}
// c.  A K scale of zero makes every score 0; it must not make -inf * 0 of a
// masked one.
template <bool FP8>
__device__ __forceinline__ float score_factor(const Args& a) {
  return FP8 ? fmaxf(a.scale_log2 * *a.k_scale, 0x1p-120f) : a.scale_log2;
}
// Factor of a row's sums for its output; a row that saw no key gives zeros.
template <bool FP8>
__device__ __forceinline__ float output_factor(const Args& a, float l) {
  return l > 0.0f ? (FP8 ? *a.v_scale : 1.0f) / l : 0.0f;
}

template <bool HALF>
__device__ __forceinline__ unsigned pack2(float x, float y) {
  const f32x2 p = {x, y};
  if constexpr (HALF) return __builtin_bit_cast(unsigned, __builtin_convertvector(p, half2_t));
  else return __builtin_bit_cast(unsigned, __builtin_convertvector(p, bf16x2));
}

// ---------------------------------------------------------------- kernel

// LDS of a workgroup: two tiles of K and V, in arrays of their own so that
// reads of one need not wait for loads into another.
template <int D>
struct Lds {
  uint8_t* k0;
  uint8_t* k1;
  uint8_t* v0;
  uint8_t* v1;
};

// Workgroup `block` of the tiles: 128 rows, 4 waves of 32.  Two waves a SIMD
// at every D, so that one's exponentials run under another's products; D =
// 256 (128 registers of sums, 64 of queries) affords that with tiles of 32
// keys: 8192 tokens of 20 heads of 256 in 640 us (1.07 PFLOP/s), with one
// wave a SIMD 900 us.  A 16384-token prompt of 40 heads of 128 takes 2.53 ms
// (1.09 PFLOP/s, 43 % of the matrix peak and 73 % of what a large library
// product reaches): the matrix cores are busy 57 % of the cycles and the
// vector units 53 %, at a clock of 1.8 GHz, so products and exponentials mostly
// take turns and hardly run side by side.  Measured and not taken there: 64 rows a wave (half the LDS reads, but one wave a SIMD: 3.1
// ms), scores of the next tile taken under the exponentials of this one
// within a wave (3.0 ms, no registers left to read ahead), 32-key tiles at
// three waves a SIMD (2.55 ms; E4M3 chunks cut in two lose 6 %), raised wave
// priority around the products (no change).
template <int D, bool FP8>
__device__ __forceinline__ void tile_rows(const Args& a, int block, const Lds<D>& lds) {
  using T = Tile<D, FP8>;
  constexpr int kSteps = D / 16;          // of the first product
  constexpr int kBlocks = T::kKeys / 32;  // key blocks of a tile
  constexpr int kDb = D / 32;             // d blocks of the output
  // LDS reads are issued this many products ahead
  constexpr int kReach = D > 128 ? 2 : 4;

  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int kvh = block % a.n_kv_heads;
  const int rest = block / a.n_kv_heads;
  const int split = rest % a.splits;
  int r, level;
  if (!tile_of(a, rest / a.splits, &r, &level)) return;
  const int64_t row0 = static_cast<int64_t>(level) * kTileRows;
  const int group = static_cast<int>(a.group.d);
  const int64_t n_rows = rows_of(a, r);
  if (row0 >= n_rows || (a.few_pieces > 0 && n_rows <= a.few_rows)) return;
  const Span s = span_of(a, r, static_cast<int>(row0), kTileRows);
  const int splits = splits_of(s, a.chunk, a.splits);
  if (split >= splits) return;
  const int begin = s.start + split * a.chunk;
  const int end = split == splits - 1 ? s.hi : begin + a.chunk;

  // this lane's row, and what all and any rows of the wave see
  const int row = s.row0 + wave * 32 + col;
  const bool real = row < n_rows;
  const int token = static_cast<int>(a.group.div(real ? row : 0));
  const int head = kvh * group + (real ? row - token * group : 0);
  int see_lo = 0, see_hi = 0;
  if (real) sees(a, s, token, &see_lo, &see_hi);
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
  const float c = score_factor<FP8>(a);

  f32x16 acc[kDb];
#pragma unroll
  for (int b = 0; b < kDb; ++b) acc[b] = f32x16{};
  float m = kNegInf, l = 0.0f;

  const int32_t* table = a.table ? a.table + r * a.ld_table : nullptr;
  const int64_t head_k = kvh * a.k_head, head_v = kvh * a.v_head;
  // this lane's reads of a tile: chunk 2 i + half of K row col at ka ^ 32 i,
  // 4-key piece of V d block b at va ^ 64 b (the exchange by the row's
  // number is the same in all the rows that are a multiple of 8 further)
  const int ka = T::k_at(col, half);
  const int va = T::v_at(4 * half + ((lane & 15) >> 2), 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) +
                 8 * (lane & 1);
  Stage<D, FP8, false> xk;
  Stage<D, FP8, true> xv;
  int id = 0;                             // page of this wave's rows of the next tile
  auto look_up = [&](int key0) {
    if (table) id = page_of(a, table, group_at<T::kRows>(s.hi, key0 + wave * T::kRows));
  };
  auto place = [&](int key0) {
    return place_of<T::kRows>(a, s, head_k, head_v, key0 + wave * T::kRows, id);
  };
  // E4M3 at D = 256 has registers for one of K and V in flight: V follows K
  constexpr bool kOneByOne = FP8 && D > 128;

  // One tile, its keys in (lk, lv); the next one's go to (nk, nv).
  auto step = [&](const uint8_t* lk, const uint8_t* lv, uint8_t* nk, uint8_t* nv, int key0) {
    const bool more = key0 + T::kKeys < end;
    const bool seen = key0 < any_hi && key0 + T::kKeys > any_lo;      // by some row of the wave
    Place p = {};
    if (more) {
      p = place(key0 + T::kKeys);
      xk.load(p, static_cast<int>(a.k_token), wave, nk);
      if constexpr (!kOneByOne) xv.load(p, static_cast<int>(a.v_token), wave, nv);
    }
    f32x16 sc[kBlocks];
    if (seen) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const bf16x8 kf = *reinterpret_cast<const bf16x8*>(lk + (ka ^ (32 * i)) + 32 * b * D * 2);
          sc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[i], i ? sc[b] : f32x16{}, 0, 0, 0);
        }
      order<0x100, kReach>();
#pragma unroll
      for (int i = 0; i < kBlocks * kSteps - kReach; ++i) {
        order<0x008, 1>();
        order<0x100, 1>();
      }
      order<0x008, kReach>();
    }
    if constexpr (kOneByOne) {
      if (more) {
        xk.store(nk, wave);
        xv.load(p, static_cast<int>(a.v_token), wave, nv);
      }
    }
    // a scalar load in flight makes LDS waits full ones: here no reads are
    look_up(key0 + 2 * T::kKeys);
    if (seen) {
      if (key0 < all_lo || key0 + T::kKeys > all_hi) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            // see_lo <= j < see_hi in one comparison
            const unsigned j = key0 + 4 * half - see_lo + (32 * b + 8 * (i >> 2) + (i & 3));
            if (j >= static_cast<unsigned>(see_hi - see_lo)) sc[b][i] = kNegInf;
          }
      }
      float top = sc[0][0];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[b][i]);
      top = half_max(top) * c;
      if (__any(top > m + kSlack)) {
        const float f = moved(&m, top);
        l *= f;
#pragma unroll
        for (int b = 0; b < kDb; ++b) acc[b] *= f;
      }
      const float shift = shift_of<FP8>(m);
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
#pragma unroll
        for (int b = 0; b < kDb; ++b) {
          const uint8_t* vp = lv + (va ^ (64 * b)) + 16 * t * D * 2;
          const s16x4 w0 = read_tr(vp);
          const s16x4 w1 = read_tr(vp + 8 * D * 2);
          const s16x8 vf = __builtin_shufflevector(w0, w1, 0, 1, 2, 3, 4, 5, 6, 7);
          if constexpr (FP8)
            acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                __builtin_bit_cast(half8_t, vf), __builtin_bit_cast(half8_t, pf), acc[b], 0, 0, 0);
          else
            acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                __builtin_bit_cast(bf16x8, vf), __builtin_bit_cast(bf16x8, pf), acc[b], 0, 0, 0);
        }
      }
      order<0x100, 2 * kReach>();
#pragma unroll
      for (int i = 0; i < T::kKeys / 16 * kDb - kReach; ++i) {
        order<0x008, 1>();
        order<0x100, 2>();
      }
      order<0x008, kReach>();
    }
    if (more) {
      if constexpr (!kOneByOne) xk.store(nk, wave);
      xv.store(nv, wave);
    }
    tile_barrier();
  };

  if (begin < end) {
    look_up(begin);
    const Place p = place(begin);
    xk.load(p, static_cast<int>(a.k_token), wave, lds.k0);
    xv.load(p, static_cast<int>(a.v_token), wave, lds.v0);
    look_up(begin + T::kKeys);
    xk.store(lds.k0, wave);
    xv.store(lds.v0, wave);
    tile_barrier();
    for (int key0 = begin; key0 < end; key0 += 2 * T::kKeys) {
      step(lds.k0, lds.v0, lds.k1, lds.v1, key0);
      if (key0 + T::kKeys < end) step(lds.k1, lds.v1, lds.k0, lds.v0, key0 + T::kKeys);
    }
  }
  l = half_sum(l);
  if (!real) return;
  const int64_t out_row = static_cast<int64_t>(s.token0) + token;
  if (splits == 1) {
    const float inv = output_factor<FP8>(a, l);
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
    const int64_t at = tile_slot(a, split, out_row, head);
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

// ------------------------------------------------- requests of few rows

// value over the four lanes that share a column of a 16x16 product
__device__ __forceinline__ float quad_max(float x) {
  unsigned u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}
__device__ __forceinline__ float quad_sum(float x) {
  unsigned u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return half_sum(__uint_as_float(r[0]) + __uint_as_float(r[1]));
}

// Keys and values of 32 keys of one wave, in flight.  K goes straight to the
// layout of the A operand (lane: key lane & 15, 16 bytes at chunk 4 i + lane
// / 16; of E4M3 codes the two halves of a chunk belong to two steps, and Q
// is read in the same order); V is read row by row for the transposing LDS.
template <int D, bool FP8>
struct Stream {
  static constexpr int kKeys = 32;
  static constexpr int kChunks = D * (FP8 ? 1 : 2) / 16;
  static constexpr int kK = kChunks / 4;                    // loads of 16 keys
  static constexpr int kV = kKeys * kChunks / 64;           // loads of the tile
  u32x4 k[2][kK], v[kV];
  Place at[2];
  int kt, vt;

  // The two groups of 16 keys at key0.
  __device__ __forceinline__ void locate(const Args& a, const Span& s, int64_t head_k,
                                         int64_t head_v, int key0, const int* ids) {
    kt = static_cast<int>(a.k_token);
    vt = static_cast<int>(a.v_token);
#pragma unroll
    for (int p = 0; p < 2; ++p) at[p] = place_of<16>(a, s, head_k, head_v, key0 + 16 * p, ids[p]);
  }
  __device__ __forceinline__ static int inside(int r, const RowBounds& b) {
    r = r < b.first ? b.first : r;
    return r > b.end ? b.end : r;
  }
  __device__ __forceinline__ void load_k() {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int row = inside(lane & 15, at[p].rows) * kt + (lane >> 4) * 16;
#pragma unroll
      for (int i = 0; i < kK; ++i) k[p][i] = load16b<true>(at[p].k, row + i * 64);
    }
  }
  __device__ __forceinline__ void load_v() {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int p = i * 64 / kChunks / 16;                  // a load lies in one group
      const int r = (i * 64 + lane) / kChunks - 16 * p, c = (i * 64 + lane) % kChunks;
      v[i] = load16b<true>(at[p].v, inside(r, at[p].rows) * vt + c * 16);
    }
  }
  // The 8 rows that 32 lanes of a transposing read touch differ by 32 bytes.
  static __device__ __forceinline__ int v_at(int r, int c) {
    return r * (D * 2) + ((c ^ (D == 64 ? ((r >> 1) & 3) << 1 : (r & 7) << 1)) << 4);
  }
  __device__ __forceinline__ void store_v(uint8_t* lds) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int r = (i * 64 + lane) / kChunks, c = (i * 64 + lane) % kChunks;
      if constexpr (FP8) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const u32x2 v0 = widen4<true>(v[i][2 * p]), v1 = widen4<true>(v[i][2 * p + 1]);
          *reinterpret_cast<u32x4*>(lds + v_at(r, 2 * c + p)) = u32x4{v0[0], v0[1], v1[0], v1[1]};
        }
      } else {
        *reinterpret_cast<u32x4*>(lds + v_at(r, c)) = v[i];
      }
    }
  }
  // A operand of step i of the first product, key group p.
  __device__ __forceinline__ bf16x8 k_operand(int p, int i) const {
    if constexpr (FP8) {
      const u32x4 w = k[p][i >> 1];
      const u32x2 a = widen4<false>(w[2 * (i & 1)]), b = widen4<false>(w[2 * (i & 1) + 1]);
      return __builtin_bit_cast(bf16x8, u32x4{a[0], a[1], b[0], b[1]});
    } else {
      return __builtin_bit_cast(bf16x8, k[p][i]);
    }
  }
};

// A request whose rows fit one 16-column operand: a decode token with its
// group of heads, a few speculated ones.  Its keys are streamed once, each
// wave taking 32 at a time straight from memory (no barrier: V passes
// through an LDS area of the wave's own); the four waves are joined at the
// end.  Bound by the read of the keys and values: 32 requests of 32768 E4M3
// keys, 4 heads of 256, in 325 us (6.6 TB/s; 128-row tiles take 986 us), 64
// ragged requests of bf16, 16 heads of 64, in 77 us (5.3 TB/s).
template <int D, bool FP8>
__device__ __forceinline__ void few_rows(const Args& a, const Cut& cut, int piece, int kvh,
                                         const Lds<D>& lds, float (*lds_m)[16], float (*lds_l)[16]) {
  using S = Stream<D, FP8>;
  constexpr int kSteps = D / 32;
  constexpr int kDb = D / 16;
  // a wave's V, and later its 16 rows of sums, in an array of its own
  static_assert(S::kKeys * D * 2 == 16 * D * 4 && 16 * D * 4 <= Tile<D, FP8>::kBytes);

  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int r = __builtin_amdgcn_readfirstlane(request_of(a, cut, piece));
  const int split = piece - first_piece(a, cut, r);
  const int group = static_cast<int>(a.group.d);
  const Span s = span_of(a, r, 0, kFewRows);
  const int64_t n_rows = static_cast<int64_t>(s.n_new) * group;
  if (n_rows < 1 || n_rows > a.few_rows) return;
  const int splits = splits_of(s, cut.chunk, a.few_chunk ? a.few_splits : 0x7FFFFFFF);
  if (split >= splits) return;
  const int begin = s.start + split * cut.chunk;
  const int end = split == splits - 1 ? s.hi : begin + cut.chunk;

  const bool real = col < n_rows;
  const int token = static_cast<int>(a.group.div(real ? col : 0));
  const int head = kvh * group + (real ? col - token * group : 0);
  int see_lo = 0, see_hi = 0;
  if (real) sees(a, s, token, &see_lo, &see_hi);

  bf16x8 qf[kSteps];
  {
    const uint8_t* qp = a.q + (static_cast<int64_t>(s.token0) + token) * a.q_token + head * a.q_head;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      // the chunk order of k_operand
      const int at = FP8 ? (i >> 1) * 128 + quad * 32 + (i & 1) * 16 : i * 64 + quad * 16;
      qf[i] = *reinterpret_cast<const bf16x8*>(qp + at);
    }
  }
  const float c = score_factor<FP8>(a);

  f32x4 acc[kDb];
#pragma unroll
  for (int b = 0; b < kDb; ++b) acc[b] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = kNegInf, l = 0.0f;

  const int32_t* table = a.table ? a.table + r * a.ld_table : nullptr;
  const int64_t head_k = kvh * a.k_head, head_v = kvh * a.v_head;
  uint8_t* lv = wave == 0 ? lds.k0 : wave == 1 ? lds.k1 : wave == 2 ? lds.v0 : lds.v1;
  S st;
  int ids[2] = {0, 0};                 // pages of the next tile's two groups
  auto look_up = [&](int key0) {
    if (!table) return;
#pragma unroll
    for (int p = 0; p < 2; ++p) ids[p] = page_of(a, table, group_at<16>(s.hi, key0 + 16 * p));
  };
  int key0 = begin + wave * S::kKeys;
  constexpr int kStride = 4 * S::kKeys;
  if (key0 < end) {
    look_up(key0);
    st.locate(a, s, head_k, head_v, key0, ids);
    st.load_k();
    st.load_v();
    if (key0 + kStride < end) look_up(key0 + kStride);
  }
  for (; key0 < end; key0 += kStride) {
    const bool more = key0 + kStride < end;
    f32x4 sc[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      sc[p] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
        sc[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(st.k_operand(p, i), qf[i], sc[p], 0, 0, 0);
    }
    st.store_v(lv);
    if (more) {
      st.locate(a, s, head_k, head_v, key0 + kStride, ids);
      st.load_k();
      st.load_v();
      if (key0 + 2 * kStride < end) look_up(key0 + 2 * kStride);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = key0 + 16 * p + 4 * quad + i;
        if (j < see_lo || j >= see_hi) sc[p][i] = kNegInf;
      }
    float top = fmaxf(fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[0][2], sc[0][3])),
                      fmaxf(fmaxf(sc[1][0], sc[1][1]), fmaxf(sc[1][2], sc[1][3])));
    top = quad_max(top) * c;
    if (__any(top > m + kSlack)) {
      const float f = moved(&m, top);
      l *= f;
#pragma unroll
      for (int b = 0; b < kDb; ++b) acc[b] *= f;
    }
    const float shift = shift_of<FP8>(m);
    u32x4 pf;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float p0 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[p][i], c, -shift));
        const float p1 = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[p][i + 1], c, -shift));
        l += p0 + p1;
        pf[2 * p + (i >> 1)] = pack2<FP8>(p0, p1);
      }
    const int vr = 4 * quad + (col >> 2);
#pragma unroll
    for (int b = 0; b < kDb; ++b) {
      const int vc = 2 * b + ((lane & 3) >> 1);
      const s16x4 v0 = read_tr(lv + S::v_at(vr, vc) + 8 * (lane & 1));
      const s16x4 v1 = read_tr(lv + S::v_at(vr + 16, vc) + 8 * (lane & 1));
      const s16x8 vf = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
      if constexpr (FP8)
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, vf),
                                                        __builtin_bit_cast(half8_t, pf), acc[b], 0, 0, 0);
      else
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, vf),
                                                         __builtin_bit_cast(bf16x8, pf), acc[b], 0, 0, 0);
    }
  }
  // join the waves: rows of sums in LDS, 16-byte pieces exchanged by row
  l = quad_sum(l);
  if (quad == 0) {
    lds_m[wave][col] = m;
    lds_l[wave][col] = l;
  }
#pragma unroll
  for (int b = 0; b < kDb; ++b)
    *reinterpret_cast<f32x4*>(lv + col * (D * 4) + (((4 * b + quad) ^ col) << 4)) = acc[b];
  __syncthreads();
  const int row = threadIdx.x >> 4, place = threadIdx.x & 15;
  if (row >= n_rows) return;
  float w[4], mm = kNegInf, ll = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lds_l[i][row] > 0.0f) mm = fmaxf(mm, lds_m[i][row]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = lds_l[i][row] > 0.0f ? __builtin_amdgcn_exp2f(lds_m[i][row] - mm) : 0.0f;
    ll = __builtin_fmaf(lds_l[i][row], w[i], ll);
  }
  const int out_token = static_cast<int>(a.group.div(row));
  const int out_head = kvh * group + row - out_token * group;
  const int64_t at = few_slot(a, piece, kvh, row);
  const float inv = output_factor<FP8>(a, ll);
  uint8_t* op = a.out + (static_cast<int64_t>(s.token0) + out_token) * a.out_token + out_head * a.out_head;
#pragma unroll
  for (int e = 0; e < D / 64; ++e) {
    const int ch = place + 16 * e;
    f32x4 o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* part = i == 0 ? lds.k0 : i == 1 ? lds.k1 : i == 2 ? lds.v0 : lds.v1;
      const f32x4 p = *reinterpret_cast<const f32x4*>(part + row * (D * 4) + ((ch ^ row) << 4));
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] = __builtin_fmaf(p[x], w[i], o[x]);
    }
    if (splits == 1) {
      const u32x2 packed = {pack2<false>(o[0] * inv, o[1] * inv), pack2<false>(o[2] * inv, o[3] * inv)};
      *reinterpret_cast<u32x2*>(op + ch * 8) = packed;
    } else {
      *reinterpret_cast<f32x4*>(a.part + at * D + ch * 4) = o;
    }
  }
  if (splits > 1 && place == 0) *reinterpret_cast<f32x2*>(a.part_ml + at * 2) = f32x2{mm, ll};
}

// Tiles of rows, requests of few rows, or both in one launch (the first
// workgroups are the tiles'), so that a step of chunks and decodes has the
// matrix work and the reads of the decodes side by side.
template <int D, bool FP8, bool TILES, bool FEW>
__global__ void __launch_bounds__(256, !TILES && D > 128 && !FP8 ? 1 : 2) attention_kernel(Args a) {
  constexpr int kBytes = TILES ? Tile<D, FP8>::kBytes : 16 * D * 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds_k0[kBytes], lds_k1[kBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t lds_v0[kBytes], lds_v1[kBytes];
  const Lds<D> lds = {lds_k0, lds_k1, lds_v0, lds_v1};
  const int block = static_cast<int>(blockIdx.x);
  if constexpr (TILES) {
    if (!FEW || block < a.tile_blocks) {
      tile_rows<D, FP8>(a, block, lds);
      return;
    }
  }
  if constexpr (FEW) {
    __shared__ float lds_m[4][16], lds_l[4][16];
    const int unit = TILES ? block - a.tile_blocks : block;
    const Cut cut = cut_of<D>(a);
    if (unit < cut.pieces * a.n_kv_heads)
      few_rows<D, FP8>(a, cut, unit / a.n_kv_heads, unit % a.n_kv_heads, lds, lds_m, lds_l);
  }
}

// Joins the chunks of each row, in chunk order within each of WAVES waves
// (one, or four for rows of many chunks: the reads of the chunks' sums are
// what takes time) and then over the waves.
template <int D, bool FP8, int WAVES>
__global__ void __launch_bounds__(256) combine_kernel(Args a) {
  constexpr int kEach = D / 64;
  __shared__ float lds_o[WAVES > 1 ? WAVES * D : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int mine = WAVES > 1 ? wave : 0;            // of the row's waves
  const int64_t row = WAVES > 1 ? static_cast<int64_t>(blockIdx.x)
                                : static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (row >= static_cast<int64_t>(a.n_tokens) * a.n_heads) return;
  const int t = static_cast<int>(row / a.n_heads), head = static_cast<int>(row % a.n_heads);
  const int r = __builtin_amdgcn_readfirstlane(find_request<true>(a, t));
  const int group = static_cast<int>(a.group.d);
  const int token0 = clampi(a.cu[r], 0, a.n_tokens);
  const int token1 = clampi(a.cu[r + 1], token0, a.n_tokens);
  if (t < token0 || t >= token1) return;             // a row of no request
  const int kvh = static_cast<int>(a.group.div(static_cast<unsigned>(head)));
  const int in_request = (t - token0) * group + head - kvh * group;
  const bool few = a.few_pieces > 0 && static_cast<int64_t>(token1 - token0) * group <= a.few_rows;
  if (!few && a.tiles == 0) return;                  // more new tokens than the caller's bound
  int splits;
  int64_t at, step;
  if (few) {
    const Cut cut = cut_of<D>(a);
    splits = splits_of(span_of(a, r, 0, kFewRows), cut.chunk, a.few_chunk ? a.few_splits : 0x7FFFFFFF);
    const int piece = first_piece(a, cut, r);
    at = few_slot(a, piece, kvh, in_request);
    step = few_slot(a, piece + 1, kvh, in_request) - at;
  } else {
    splits = splits_of(span_of(a, r, in_request & -kTileRows, kTileRows), a.chunk, a.splits);
    at = tile_slot(a, 0, t, head);
    step = tile_slot(a, 1, t, head) - at;
  }
  if (splits == 1) return;
  typedef float vec __attribute__((ext_vector_type(kEach)));
  if constexpr (WAVES == 1) {
    constexpr int kShort = 8;
    if (splits <= kShort) {
      // all reads at once
      f32x2 ml = {kNegInf, 0.0f};
      if (lane < splits) ml = *reinterpret_cast<const f32x2*>(a.part_ml + (at + lane * step) * 2);
      vec x[kShort];
#pragma unroll
      for (int i = 0; i < kShort; ++i)
        x[i] = i < splits ? *reinterpret_cast<const vec*>(a.part + (at + i * step) * D + lane * kEach)
                          : vec{};
      float m = ml[1] > 0.0f ? ml[0] : kNegInf;
#pragma unroll
      for (int off = 1; off < kShort; off <<= 1) m = fmaxf(m, __shfl_xor(m, off));
      const float f = ml[1] > 0.0f ? __builtin_amdgcn_exp2f(ml[0] - m) : 0.0f;
      float l = 0.0f;
      vec o = {};
#pragma unroll
      for (int i = 0; i < kShort; ++i) {
        const float fi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), i));
        l = __builtin_fmaf(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ml[1]), i)), fi, l);
#pragma unroll
        for (int e = 0; e < kEach; ++e) o[e] = __builtin_fmaf(x[i][e], fi, o[e]);
      }
      const float inv = output_factor<FP8>(a, l);
      __bf16* op = reinterpret_cast<__bf16*>(a.out + t * a.out_token + head * a.out_head) + lane * kEach;
#pragma unroll
      for (int e = 0; e < kEach; ++e) op[e] = static_cast<__bf16>(o[e] * inv);
      return;
    }
  }
  // a lane takes the bound and the sum of weights of every 64th chunk
  float m = kNegInf;
  for (int i = lane; i < splits; i += 64) {
    const f32x2 ml = *reinterpret_cast<const f32x2*>(a.part_ml + (at + i * step) * 2);
    if (ml[1] > 0.0f) m = fmaxf(m, ml[0]);
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) m = fmaxf(m, __shfl_xor(m, off));
  float l = 0.0f, o[kEach] = {};
  for (int i0 = 0; i0 < splits; i0 += 64) {
    float f = 0.0f;
    if (i0 + lane < splits) {
      const f32x2 ml = *reinterpret_cast<const f32x2*>(a.part_ml + (at + (i0 + lane) * step) * 2);
      f = ml[1] > 0.0f ? __builtin_amdgcn_exp2f(ml[0] - m) : 0.0f;
      l = __builtin_fmaf(ml[1], f, l);
    }
    const int n = splits - i0 < 64 ? splits - i0 : 64;
    const float* p = a.part + (at + i0 * step) * D + lane * kEach;
#pragma unroll 8
    for (int i = mine; i < n; i += WAVES) {
      const float fi = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f), i));
      const vec x = *reinterpret_cast<const vec*>(p + i * step * D);
#pragma unroll
      for (int e = 0; e < kEach; ++e) o[e] = __builtin_fmaf(x[e], fi, o[e]);
    }
  }
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) l += __shfl_xor(l, off);
  if constexpr (WAVES > 1) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) lds_o[wave * D + lane * kEach + e] = o[e];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      o[e] = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) o[e] += lds_o[w * D + lane * kEach + e];
    }
  }
  const float inv = output_factor<FP8>(a, l);
  __bf16* op = reinterpret_cast<__bf16*>(a.out + t * a.out_token + head * a.out_head) + lane * kEach;
#pragma unroll
  for (int e = 0; e < kEach; ++e) op[e] = static_cast<__bf16>(o[e] * inv);
}

// ------------------------------------------------------------------ host

constexpr int64_t kCus = 256;
// Requests too many to be planned by the kernel even out by number, and only
// those far longer than most are cut: pieces of at least kLongest keys, at most
// kMostPieces (of a request and a head) by the bound of the lengths, so that
// neither the empty ones nor the workspace grow with it.  257 requests of
// 1000 E4M3 keys, 5 rows, 8 heads of 128, called with a bound of 131072: 98
// us and 15 MiB in 6168 pieces, 261 us and 163 MiB in pieces of kLongest keys
// however many that makes.  One of 131072 keys among 256 of 2048: 525 us,
// uncut 1269 us, twice as many pieces 346 us (but 512 requests of 4 heads of
// 256, one of them of 65536 keys: 559 us, twice as many pieces 957 us).
constexpr int64_t kLongest = 4096;
constexpr int64_t kMostPieces = 8192;

struct Plan {
  int64_t tiles, splits, chunk;           // tiles == 0: no request of many rows
  // few_pieces == 0: none of few rows; few_chunk == 0: cut by the kernel
  int64_t few_rows, few_pieces, few_chunk, few_splits;
  int64_t slots;                          // places of chunks' sums
};

// Keys that the first and last of `tokens` neighbours see together, with a
// window the first 16-key group rounded down included.
int64_t span_keys(const AttnCall& c, int64_t tokens) {
  const int64_t keys = c.table ? c.max_kv : c.max_new;
  if (!c.window) return keys;
  const int64_t seen = c.window + tokens - 1;
  return (c.causal && keys > seen ? seen : keys) + 15;
}

// Chunks of the tiles' keys by their estimated time.  Two workgroups fit a
// CU, so `tiles` of them run in rounds of 512; a last round of less than
// half takes about 0.62 of one (a workgroup alone on its CU is faster).
// Cutting the keys evens the rounds out but writes and reads each chunk's
// sums.  Uncut, in 2, 3 and 4 chunks, with what the estimate takes in brackets:
// 2048 tokens of 40 heads over 32001 E4M3 keys, 1.25 rounds: 1556, 1362,
// [1388], 1338 us; the same over bf16 keys: 1438, 1297, [1324], 1302; 512
// tokens over 16384 keys: 311, 233, [187], 215; 3 chunks and 21 decodes: 194, 118,
// 88, [79]; 7 prompts of up to 2001 tokens: [99], 151, 128, 192; a prompt of
// 16384: [2526], 3599, 2990, 4239; 8192 tokens, all keys: [1277], 1423, 1490,
// 1544.  Rates: 1 PFLOP/s, 4 TB/s for the sums, 6 us a launch.  Cut workgroups
// fill at most kMostRounds rounds, which bounds the workspace: beyond that the
// rounds are even enough and only the sums are left (8192 tokens over 32768
// keys, 5 rounds: 4.46 ms uncut, 4.80 in 2 and 5.0 in 3 chunks; over 131072
// keys 19.9 ms uncut, 20.8 in 2 and 21.7 in 6, with 975 MiB of sums).  3500
// tokens over 65536 keys, 2.1 rounds: 4.90 ms uncut, 4.65 in the 3 chunks that
// this still allows.
constexpr double kMostRounds = 7.0;
void cut_tiles(const AttnCall& c, int64_t group, Plan* p) {
  const int64_t keys = span_keys(c, kTileRows / group + 2);
  const double wgs = (static_cast<double>(c.n_tokens) * group / kTileRows + 0.5 * c.n_requests) *
                     c.n_kv_heads;
  // rows that see from none to all of the keys even out by themselves (the
  // longest are first)
  const bool graded = c.causal && (!c.table || c.max_kv < 2 * c.max_new);
  const double round_us = 2.0 * kCus * kTileRows * keys * 4.0 * c.d / 1e9;
  const double sums_us = static_cast<double>(c.n_tokens) * c.n_heads * c.d * 8.0 / 4e6;
  double best = 0.0;
  int64_t splits = 1;
  for (int64_t n = 1; n <= 16 && (n == 1 || (keys >= 256 * n && wgs * n <= 2.0 * kCus * kMostRounds)); ++n) {
    const double r = wgs * n / (2.0 * kCus), full = floor(r);
    const double rounds = graded && r > 1.0 ? r : full + (r - full > 0.5 ? 1.0 : r > full ? 0.62 : 0.0);
    const double us = round_us * rounds / n + (n > 1 ? 6.0 + n * sums_us : 0.0);
    if (n == 1 || us < best) {
      best = us;
      splits = n;
    }
  }
  p->chunk = (keys + splits * 128 - 1) / (splits * 128) * 128;
  if (p->chunk < 128) p->chunk = 128;
  p->splits = (keys + p->chunk - 1) / p->chunk;
  if (p->splits < 1) p->splits = 1;
}

Plan plan_of(const AttnCall& c) {
  Plan p = {};
  const int64_t group = c.n_heads / c.n_kv_heads;
  const bool many = !c.table || c.max_new * group > kFewRows;
  // a prompt of few rows has few keys too: its tile costs no more; and a
  // single request of many rows has none of few next to it
  const bool few = c.table && group <= kFewRows && !(many && c.n_requests == 1);
  if (many) {
    p.tiles = c.n_tokens * group / kTileRows + c.n_requests;
    cut_tiles(c, group, &p);
  }
  if (few) {
    p.few_rows = many ? kFewRows : c.max_new * group;
    const int64_t keys = span_keys(c, kFewRows), least = few_least(static_cast<int>(c.d));
    if (c.n_requests == 1 && keys > least) {
      // its length is the bound: enough pieces for every CU
      const int64_t want = (4 * kCus + c.n_kv_heads - 1) / c.n_kv_heads;
      p.few_chunk = ((keys + want - 1) / want + 127) / 128 * 128;
      if (p.few_chunk < least) p.few_chunk = least;
      p.few_splits = p.few_pieces = (keys + p.few_chunk - 1) / p.few_chunk;
    } else if (c.n_requests <= kPlanned && keys > least) {
      p.few_pieces = pieces_bound(c.n_requests, c.n_kv_heads);
    } else {
      // short keys are not cut; of very many requests only long ones are
      p.few_splits = c.n_requests <= kPlanned ? 1 : (keys + kLongest - 1) / kLongest;
      const int64_t most = kMostPieces / (c.n_requests * c.n_kv_heads);
      if (p.few_splits > most) p.few_splits = most;
      if (p.few_splits < 1) p.few_splits = 1;
      p.few_chunk = ((keys + p.few_splits - 1) / p.few_splits + 127) / 128 * 128;
      if (p.few_chunk < 128) p.few_chunk = 128;
      p.few_pieces = c.n_requests * p.few_splits;
    }
  }
  if (p.splits > 1) p.slots += p.splits * c.n_tokens * c.n_heads;
  if (p.few_splits != 1) p.slots += p.few_pieces * c.n_kv_heads * p.few_rows;
  return p;
}

template <int D, bool FP8>
void launch(const Args& a, hipStream_t stream) {
  const unsigned tiles = static_cast<unsigned>(a.tile_blocks), few = static_cast<unsigned>(a.few_blocks);
  if (tiles && few) attention_kernel<D, FP8, true, true><<<tiles + few, 256, 0, stream>>>(a);
  else if (tiles) attention_kernel<D, FP8, true, false><<<tiles, 256, 0, stream>>>(a);
  else if (few) attention_kernel<D, FP8, false, true><<<few, 256, 0, stream>>>(a);
  if (a.splits > 1 || (a.few_pieces > 0 && a.few_splits != 1)) {
    // four waves a row for many chunks, as long as the rows are few: one request
    // of 6000 keys (20 rows, d 256) 18 us with four and 20 with one, 64 ragged
    // ones of up to 4000 (1024 rows, d 64) 36 and 38 us, 256 of 1500 (10240
    // rows, d 128) 158 and 138 us.  Between about 2000 rows and the bound one
    // wave is the faster too (200 ragged requests, 3200 to 8000 rows: by 4 to
    // 18 %).  A step of chunks and decodes, 7220 rows of mostly three chunks,
    // takes one: 79 us, with four 84
    const int64_t rows = static_cast<int64_t>(a.n_tokens) * a.n_heads;
    if ((!tiles || a.splits > 8) && rows <= 8192)
      combine_kernel<D, FP8, 4><<<static_cast<unsigned>(rows), 256, 0, stream>>>(a);
    else
      combine_kernel<D, FP8, 1><<<static_cast<unsigned>((rows + 3) / 4), 256, 0, stream>>>(a);
  }
}

}  // namespace

// Enough for either mask: the plan depends on it, the callers' query does not.
int64_t attention_workspace(const AttnCall& c) {
  AttnCall other = c;
  other.causal = !c.causal;
  const int64_t a = plan_of(c).slots, b = plan_of(other).slots;
  return (a > b ? a : b) * (c.d + 2) * 4;
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
  a.part_ml = a.part + p.slots * c.d;
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
  a.tile_blocks = static_cast<int>(p.tiles * p.splits * c.n_kv_heads);
  a.chunk = static_cast<int>(p.chunk);
  a.few_rows = static_cast<int>(p.few_rows);
  a.few_pieces = static_cast<int>(p.few_pieces);
  a.few_chunk = static_cast<int>(p.few_chunk);
  a.few_splits = static_cast<int>(p.few_splits);
  a.few_blocks = static_cast<int>(p.few_pieces * c.n_kv_heads);
  const bool fp8 = paged && c.pool.fp8;
  if (c.d == 64) fp8 ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
  else if (c.d == 128) fp8 ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
  else fp8 ? launch<256, true>(a, stream) : launch<256, false>(a, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
