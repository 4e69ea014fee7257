// Y = A B^T on MXFP4 operands for gfx950.
//
// The 4-bit matrix instructions take E2M1 operands with one E8M0 scale per 32
// elements of K, which is the format as it is stored: a lane's operand is 16
// bytes of codes (one block) of its row and the block's scale byte, and
// nothing is decoded.  Products and scales are exact; sums are binary32.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "gemm_common.h"
#include "internal.h"
#include "mxfp4_plan.h"

namespace nvfp4 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ unsigned short bf16_bits(float f) {
  return __builtin_bit_cast(unsigned short, static_cast<__bf16>(f));
}

__device__ __forceinline__ unsigned bf16_pair(float a, float b) {
  const bf16x2 p = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(unsigned, p);
}

__device__ __forceinline__ i32x8 operand(u32x4 c) {
  return {static_cast<int>(c[0]), static_cast<int>(c[1]), static_cast<int>(c[2]),
          static_cast<int>(c[3]), 0, 0, 0, 0};
}

// 16 x 16 outputs, 128 of K; scales in byte 0
__device__ __forceinline__ f32x4 product16(u32x4 a, unsigned sa, u32x4 b, unsigned sb, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a), operand(b), c, 4, 4, 0,
                                                          static_cast<int>(sa), 0,
                                                          static_cast<int>(sb));
}

// 32 x 32 outputs, 64 of K; scales in byte 0 (STEP 0) or 2 (STEP 1)
template <int STEP>
__device__ __forceinline__ f32x16 product(u32x4 a, unsigned sa, u32x4 b, unsigned sb, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(a), operand(b), c, 4, 4, 2 * STEP,
                                                         static_cast<int>(sa), 2 * STEP,
                                                         static_cast<int>(sb));
}

// ---------------------------------------------------------------------------
// Streaming kernel: one operand (L) of at most 64 rows, the other (S) read once; or
// L in groups of 64 rows, for small products of a long K.
//
// A workgroup of NW waves takes SF 16 rows of S and LF 16 rows of L, the waves a
// part of K each.  Operands go from memory straight to registers: a
// wave has the loads of up to eight k-steps (128 of K) in flight at once, for K
// up to 8192 mostly all that it needs, and L comes from L2.  The waves' sums meet in
// LDS and are added in a fixed order.  What bounds it is the latency of one
// round of loads and the reduction behind it.
//
// Lane l of a k-step has row l % 16 and block l / 16 of the four; its scale byte
// comes with those of its row, four k-steps in one load, or (RAGGED: k no
// multiple of 128) by itself.  Rows past the last read the last; blocks past k
// lie beyond the resource's range and are zeros.
template <int F, int STEPS, bool RAGGED>
struct StreamOperand {
  __amdgpu_buffer_rsrc_t codes, scales;
  unsigned code_off[F], scale_off[F];
  u32x4 code[F][STEPS];
  u32x4 scale[F][RAGGED ? STEPS : STEPS / 4];    // RAGGED: one byte each

  __device__ __forceinline__ void init(const uint8_t* c, const uint8_t* s, int64_t row0,
                                       int64_t rows, int64_t k, int lane) {
    const unsigned kbytes = static_cast<unsigned>(k / 2), blocks = static_cast<unsigned>(k / 32);
    const int last = static_cast<int>(rows - 1 - row0 < F * 16 - 1 ? rows - 1 - row0 : F * 16 - 1);
    codes = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(c + row0 * kbytes), 0,
                                              static_cast<int>((last + 1) * kbytes), 0x00020000);
    scales = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(s + row0 * blocks), 0,
                                               static_cast<int>((last + 1) * blocks), 0x00020000);
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int row = f * 16 + (lane & 15);
      code_off[f] = static_cast<unsigned>(row < last ? row : last) * kbytes + (lane >> 4) * 16;
      scale_off[f] = static_cast<unsigned>(row < last ? row : last) * blocks;
    }
  }

  // k-steps [first, first + n), n <= STEPS
  __device__ __forceinline__ void load(int first, int n, int blocks, int lane) {
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int block = 4 * (first + i) + (lane >> 4);
      const bool in = i < n && (!RAGGED || block < blocks);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        code[f][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
            codes, in ? code_off[f] + (first + i) * 64 : 0x80000000u, 0, 0));
        if constexpr (RAGGED)
          scale[f][i][0] = __builtin_amdgcn_raw_buffer_load_b8(
              scales, in ? scale_off[f] + block : 0x80000000u, 0, 0);
      }
    }
    if constexpr (!RAGGED) {
#pragma unroll
      for (int i = 0; i < STEPS / 4; ++i)
#pragma unroll
        for (int f = 0; f < F; ++f)
          scale[f][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
              scales, 4 * i < n ? scale_off[f] + (first + 4 * i) * 4 : 0x80000000u, 0, 0));
    }
  }

  __device__ __forceinline__ unsigned scale_of(int f, int i, int lane) const {
    if constexpr (RAGGED) return scale[f][i][0];
    else return scale[f][i / 4][i % 4] >> (8 * (lane >> 4));
  }
};

template <int NW, int SF, int LF, bool RAGGED, bool S_IS_B, int OUT>
__global__ void __launch_bounds__(NW * 64)
mxfp4_gemm_stream(const uint8_t* __restrict__ s_codes, const uint8_t* __restrict__ s_scales,
                  int64_t s_rows, const uint8_t* __restrict__ l_codes,
                  const uint8_t* __restrict__ l_scales, int64_t l_rows, int64_t k,
                  void* __restrict__ out, int64_t ldo) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * (SF * 16);
  const int64_t lrow0 = static_cast<int64_t>(blockIdx.y) * (LF * 16);
  const int blocks = static_cast<int>(k / 32), steps = (blocks + 3) >> 2;
  const int from = steps * wave / NW, to = steps * (wave + 1) / NW;

  // k-steps in flight: what the registers hold
  constexpr int STEPS = SF + LF > 5 || NW < 8 ? 4 : 8;
  StreamOperand<SF, STEPS, RAGGED> so;
  StreamOperand<LF, STEPS, RAGGED> lo;
  so.init(s_codes, s_scales, row0, s_rows, k, lane);
  lo.init(l_codes, l_scales, lrow0, l_rows, k, lane);
  f32x4 acc[SF][LF] = {};
  for (int st = from; st < to; st += STEPS) {
    const int n = to - st < STEPS ? to - st : STEPS;
    so.load(st, n, blocks, lane);
    lo.load(st, n, blocks, lane);
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
      if (i < n) {
#pragma unroll
        for (int a = 0; a < SF; ++a)
#pragma unroll
          for (int b = 0; b < LF; ++b) {
            const unsigned ss = so.scale_of(a, i, lane), ls = lo.scale_of(b, i, lane);
            // B's rows down, A's across
            acc[a][b] = S_IS_B ? product16(so.code[a][i], ss, lo.code[b][i], ls, acc[a][b])
                               : product16(lo.code[b][i], ls, so.code[a][i], ss, acc[a][b]);
          }
      }
  }

  __shared__ f32x4 sums[NW][SF * LF][64];
#pragma unroll
  for (int a = 0; a < SF; ++a)
#pragma unroll
    for (int b = 0; b < LF; ++b) sums[wave][a * LF + b][lane] = acc[a][b];
  __syncthreads();
  const bool whole = reinterpret_cast<uintptr_t>(out) % (OUT == kOutF32 ? 16 : 8) == 0 &&
                     ldo % 4 == 0;
  for (int q = threadIdx.x; q < SF * LF * 64; q += NW * 64) {
    const int tile = q >> 6, l = q & 63;
    f32x4 y = sums[0][tile][l];
#pragma unroll
    for (int w = 1; w < NW; ++w) y += sums[w][tile][l];
    // lane l of a tile: column of A's rows l % 16, four of B's from 4 (l / 16)
    const int64_t sr = row0 + tile / LF * 16, lr = lrow0 + tile % LF * 16;
    const int64_t m = (S_IS_B ? lr : sr) + (l & 15), n = (S_IS_B ? sr : lr) + (l >> 4) * 4;
    const int64_t rows_m = S_IS_B ? l_rows : s_rows, rows_n = S_IS_B ? s_rows : l_rows;
    if (m >= rows_m) continue;
    if (whole && n + 4 <= rows_n) {
      if constexpr (OUT == kOutF32)
        *reinterpret_cast<f32x4*>(static_cast<float*>(out) + m * ldo + n) = y;
      else
        *reinterpret_cast<u32x2*>(static_cast<unsigned short*>(out) + m * ldo + n) =
            u32x2{bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < rows_n) {
          if constexpr (OUT == kOutF32) static_cast<float*>(out)[m * ldo + n + i] = y[i];
          else static_cast<unsigned short*>(out)[m * ldo + n + i] = bf16_bits(y[i]);
        }
    }
  }
}

// ---------------------------------------------------------------------------
// Tiled kernel.
//
// A workgroup of WM x WN waves computes a tile of WM TM 32 rows of A by WN TN
// 32 rows of B, 256 of K a stage: 128 bytes of a row, a whole line, because L2
// answers a request of half a line in the time of a whole one (stages of 128 of
// K: the loads alone took 734 us of 32768 x 10240 x 5120's 926).  Stages go from
// memory straight to one of two slots in LDS.  A stage is four k-steps of 64; a
// wave reads the operands of a k-step while the products of the one before it
// run, so the last reads of a slot are behind the third k-step's products, and
// one wait and one barrier there free it: the stage after next goes into it
// while the fourth k-step and the next stage run.
//
// A row's eight 16-byte pieces of a stage (the eight blocks) are exchanged by an
// exclusive or with the row number, so that the operand reads of a wave fall on
// different banks.  Its scales are 8 bytes of a line of their own, so they come
// for two stages at once; every wave takes those of its rows to registers at the
// start of the two, which frees their place in LDS for the next.  Where k is no
// multiple of 128 (RAGGED) a row's scales begin at any byte: five dwords hold
// them, joined by the row's shift.  Blocks past k are read as zeros: codes
// beyond the resource's range, scales masked.
//
// The products are computed transposed (B's rows down, A's across), so that a
// lane holds four consecutive columns of one row of Y.  Tiles leave through LDS
// in whole 16-byte pieces.
//
// What bounds it is the clock that its power leaves and, in equal part, waits:
// 32768 x 10240 x 5120 on random codes 793-850 us (3.9-4.3 PFLOP/s), matrix cores
// busy 62 % of the cycles at 1.58 GHz; on constant codes, which switch less, 688 us,
// 55 % at 2.15 GHz.  LDS reads take 31 % of the cycles, waits for loads and the
// barrier 28 % of the waves' time.  A loop of the same products alone reaches
// 6.3-6.5 PFLOP/s on random codes.  Rows that are no whole lines (K = 5152: 2576
// bytes) cost a second line for each piece: 1003 x 17536 70 us at K = 5120, 89 at
// 5152.
constexpr int kBK = 256;
constexpr int kRowBytes = kBK / 2;

__device__ __forceinline__ int piece_xor(int row) { return (row >> 1) & 7; }

// One operand's loads of a wave: ROWS x 128 bytes of codes a stage, and 16 bytes
// of scales a row every two stages (a dword more if RAGGED).  Offsets are
// 32-bit, from the tile's first row; rows past the last read the last.
template <int ROWS, int NW, bool RAGGED>
struct Loads {
  static constexpr int kCodes = ROWS / 8 / NW;
  static constexpr int kPerWave = (ROWS + 64 * NW - 1) / (64 * NW);    // rows / 64 of scales
  static constexpr int kRows = kPerWave * NW * 64;                     // places in LDS
  static constexpr int kScaleBytes = kRows * (RAGGED ? 20 : 16);
  static_assert(ROWS % (16 * NW) == 0, "rows split evenly over the waves");
  __amdgpu_buffer_rsrc_t codes, scales;
  unsigned code_off[kCodes], scale_off[kPerWave];

  __device__ __forceinline__ void init(const uint8_t* c, const uint8_t* s, int64_t row0,
                                       int64_t rows, int64_t k, int wave, int lane) {
    const unsigned kbytes = static_cast<unsigned>(k / 2), blocks = static_cast<unsigned>(k / 32);
    const int last = static_cast<int>(rows - 1 - row0 < ROWS - 1 ? rows - 1 - row0 : ROWS - 1);
    const int64_t s0 = row0 * blocks, s_from = s0 & ~int64_t(3);
    codes = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(c + row0 * kbytes), 0,
                                              static_cast<int>((last + 1) * kbytes), 0x00020000);
    // whole dwords: the last may hold up to three bytes behind the scales,
    // which are not used
    scales = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(s + s_from), 0,
        static_cast<int>((s0 - s_from + (last + 1) * static_cast<int64_t>(blocks) + 3) & ~int64_t(3)),
        0x00020000);
#pragma unroll
    for (int i = 0; i < kCodes; ++i) {
      const int q = (wave * kCodes + i) * 64 + lane, row = q >> 3;
      code_off[i] = static_cast<unsigned>(row < last ? row : last) * kbytes +
                    ((q & 7) ^ piece_xor(row)) * 16;
    }
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int row = (wave * kPerWave + i) * 64 + lane;
      scale_off[i] = (static_cast<unsigned>(s0 - s_from) +
                      static_cast<unsigned>(row < last ? row : last) * blocks) & ~3u;
    }
  }

  // `left`: blocks from this stage's first to the end of K (below 8 in a last
  // stage, or past it)
  __device__ __forceinline__ void issue_codes(int stage, int left, uint8_t* lds, int wave,
                                              int lane) const {
    // a scalar offset within the resource, also where every lane's lies beyond it
    const int from = left > 0 ? stage * kRowBytes : 0;
#pragma unroll
    for (int i = 0; i < kCodes; ++i) {
      const int q = (wave * kCodes + i) * 64 + lane;
      const unsigned off = ((q & 7) ^ piece_xor(q >> 3)) < left ? code_off[i] : 0x80000000u;
      lds_buf16(codes, lds + (wave * kCodes + i) * 1024, off, from);
    }
  }

  // the scales of stages 2 window and 2 window + 1; past the end of K any, which
  // are not used
  __device__ __forceinline__ void issue_scales(int window, int blocks, uint8_t* lds, int wave) const {
    const int from = window * 16 < blocks ? window * 16 : 0;
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      lds_buf16(scales, lds + (wave * kPerWave + i) * 1024, scale_off[i], from);
      if constexpr (RAGGED)
        lds_buf4(scales, lds + kRows * 16 + (wave * kPerWave + i) * 256, scale_off[i] + 16, from);
    }
  }
};

// A wave's operands of one k-step of T tiles of 32 rows.
template <int T>
struct Operand {
  u32x4 code[T];
};

// `at`: the lane's place in the rows of its first tile (the exchange does not
// change from one tile of 32 rows to the next)
template <int T>
__device__ __forceinline__ void read_codes(Operand<T>& o, const uint8_t* lds, int at) {
#pragma unroll
  for (int t = 0; t < T; ++t)
    o.code[t] = *reinterpret_cast<const u32x4*>(lds + at + t * 32 * kRowBytes);
}

// The scales of two stages of T tiles of rows, and of them those of the U-th
// pair of k-steps as the products take them: byte 0 and byte 2 are this
// half-wave's blocks of the two.
template <int T, bool RAGGED, int ROWS>
struct Scales {
  u32x4 w[T];
  unsigned more[RAGGED ? T : 1];
  __device__ __forceinline__ void read(const uint8_t* lds, int row) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      w[t] = *reinterpret_cast<const u32x4*>(lds + row * 16 + t * 512);
      if constexpr (RAGGED)
        more[t] = *reinterpret_cast<const unsigned*>(lds + ROWS * 16 + row * 4 + t * 128);
    }
  }
  template <int U>
  __device__ __forceinline__ void take(unsigned (&s)[T], int half, const unsigned (&shift)[T],
                                       unsigned mask) const {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      s[t] = w[t][U];
      if constexpr (RAGGED)
        s[t] = __builtin_amdgcn_alignbyte(U == 3 ? more[t] : w[t][(U + 1) & 3], s[t], shift[t]);
      s[t] = (s[t] & mask) >> (half * 8);
    }
  }
};

template <int I>
struct Index {
  static constexpr int value = I;
};

// One scheduling region of products: the next operands' reads go out behind the
// first products, one by one (left to itself the compiler puts them behind all,
// to reuse registers, and the next products wait for LDS), and the loads spread
// over all of them (a burst of loads holds up the products behind it).
template <int PRODUCTS, int READS, int LOADS>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < PRODUCTS; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                   // MFMA
    if (i < READS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);    // LDS read
    if (i * LOADS / PRODUCTS != (i + 1) * LOADS / PRODUCTS)
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);                 // memory read
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <int WM, int WN, int TM, int TN, bool RAGGED>
struct TileShape {
  static constexpr int NW = WM * WN, BM = WM * TM * 32, BN = WN * TN * 32;
  using LoadsA = Loads<BM, NW, RAGGED>;
  using LoadsB = Loads<BN, NW, RAGGED>;
  static constexpr int kSlotBytes = (BM + BN) * kRowBytes;
  static constexpr int kScaleBytes = LoadsA::kScaleBytes + LoadsB::kScaleBytes;
};

template <int WM, int WN, int TM, int TN, bool RAGGED, int OUT>
__global__ void __launch_bounds__(WM * WN * 64, 1)
mxfp4_gemm_tiled(const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales,
                 int64_t m, const uint8_t* __restrict__ b_codes,
                 const uint8_t* __restrict__ b_scales, int64_t n, int64_t k,
                 void* __restrict__ out, int64_t ldo, int tiles_m, int tiles_n) {
  using S = TileShape<WM, WN, TM, TN, RAGGED>;
  // an object of its own for each slot: a fill of one slot then does not look
  // like a write to what the reads of the other wait for
  __shared__ __attribute__((aligned(1024))) uint8_t s0[S::kSlotBytes], s1[S::kSlotBytes],
      scale_lds[S::kScaleBytes];

  // workgroups are dealt to the 8 XCDs in turn: each XCD takes a contiguous
  // range of tiles, in groups of 4 tiles of rows, so that those that run
  // together share panels in its L2
  const int ntiles = tiles_m * tiles_n;
  int bid = blockIdx.x;
  if (ntiles % 8 == 0) bid = (bid % 8) * (ntiles / 8) + bid / 8;
  constexpr int kGroup = 4;
  const int first_m = bid / (kGroup * tiles_n) * kGroup;
  const int gm = min(tiles_m - first_m, kGroup);
  const int in_group = bid % (kGroup * tiles_n);
  const int64_t m0 = static_cast<int64_t>(first_m + in_group % gm) * S::BM;
  const int64_t n0 = static_cast<int64_t>(in_group / gm) * S::BN;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int arow = wave / WN * TM * 32, brow = wave % WN * TN * 32;
  const int blocks = static_cast<int>(k / 32), nk = (blocks + 7) >> 3;

  typename S::LoadsA la;
  typename S::LoadsB lb;
  la.init(a_codes, a_scales, m0, m, k, wave, lane);
  lb.init(b_codes, b_scales, n0, n, k, wave, lane);
  unsigned ashift[TM], bshift[TN];
  if constexpr (RAGGED) {
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      const int64_t row = m0 + arow + t * 32 + (lane & 31);
      ashift[t] = static_cast<unsigned>(((row < m ? row : m - 1) * blocks) & 3);
    }
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      const int64_t row = n0 + brow + t * 32 + (lane & 31);
      bshift[t] = static_cast<unsigned>(((row < n ? row : n - 1) * blocks) & 3);
    }
  }

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  constexpr int kB = S::BM * kRowBytes, kSB = S::LoadsA::kScaleBytes;
  auto issue_a = [&](int st, uint8_t* slot) { la.issue_codes(st, blocks - 8 * st, slot, wave, lane); };
  auto issue_b = [&](int st, uint8_t* slot) {
    lb.issue_codes(st, blocks - 8 * st, slot + kB, wave, lane);
  };
  auto issue_scales = [&](int window) {
    la.issue_scales(window, blocks, scale_lds, wave);
    lb.issue_scales(window, blocks, scale_lds + kSB, wave);
  };
  issue_scales(0);
  issue_a(0, s0);
  issue_b(0, s0);
  issue_a(1, s1);
  __builtin_amdgcn_s_waitcnt(kVmcntKeepOf(S::LoadsA::kCodes));
  stage_barrier();

  // places of the lane's first piece (those of the other k-steps are 32, 64
  // and 96 bytes off, exchanged) and first row
  const int h = lane >> 5, r = lane & 31;
  const int lane_at = r * kRowBytes + (h ^ piece_xor(r)) * 16;
  const int a0 = arow * kRowBytes + lane_at, b0 = kB + brow * kRowBytes + lane_at;
  Operand<TM> ca, na;
  Operand<TN> cb, nb;
  Scales<TM, RAGGED, S::LoadsA::kRows> wa;
  Scales<TN, RAGGED, S::LoadsB::kRows> wb;
  read_codes(ca, s0, a0);
  read_codes(cb, s0, b0);
  wa.read(scale_lds, arow + r);
  wb.read(scale_lds + kSB, brow + r);

  unsigned sa[TM], sb[TN];
  auto take = [&](auto index, int first) {
    // scales of blocks past k are zeros: a next row's may be a NaN
    const int left = blocks - first;
    const unsigned mask = left >= 4 ? ~0u : left > 0 ? (1u << (8 * left)) - 1u : 0u;
    wa.template take<decltype(index)::value>(sa, h, ashift, mask);
    wb.template take<decltype(index)::value>(sb, h, bshift, mask);
  };
  auto products = [&](auto step, const Operand<TM>& oa, const Operand<TN>& ob) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = product<decltype(step)::value>(ob.code[j], sb[j], oa.code[i], sa[i], acc[i][j]);
  };
  // Stage kt, in `slot`; P: the first or second of the two that share scales.
  auto stage = [&](auto index, int kt, uint8_t* slot, uint8_t* other) {
    constexpr int P = decltype(index)::value;
    take(Index<2 * P>(), 8 * kt);
    issue_b(kt + 1, other);
    read_codes(na, slot, a0 ^ 32);
    read_codes(nb, slot, b0 ^ 32);
    products(Index<0>(), ca, cb);
    interleave<TM * TN, TM + TN, S::LoadsB::kCodes>();
    read_codes(ca, slot, a0 ^ 64);
    read_codes(cb, slot, b0 ^ 64);
    products(Index<1>(), na, nb);
    interleave<TM * TN, TM + TN, 0>();
    take(Index<2 * P + 1>(), 8 * kt + 4);
    read_codes(na, slot, a0 ^ 96);
    read_codes(nb, slot, b0 ^ 96);
    products(Index<0>(), ca, cb);
    interleave<TM * TN, TM + TN, 0>();
    // this wave has read all of this slot, and its loads of the next stage
    // have landed
    __builtin_amdgcn_s_waitcnt(0);
    stage_barrier();
    if constexpr (P == 0) issue_scales((kt >> 1) + 1);
    issue_a(kt + 2, slot);
    read_codes(ca, other, a0);
    read_codes(cb, other, b0);
    if constexpr (P == 1) {
      wa.read(scale_lds, arow + r);
      wb.read(scale_lds + kSB, brow + r);
    }
    products(Index<1>(), na, nb);
    interleave<TM * TN, TM + TN, S::LoadsA::kCodes>();
  };
  int kt = 0;
  for (; kt + 2 <= nk; kt += 2) {
    stage(Index<0>(), kt, s0, s1);
    stage(Index<1>(), kt + 1, s1, s0);
  }
  if (kt < nk) stage(Index<0>(), kt, s0, s1);
  // no fill may still be writing LDS when it is used again or released
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();

  // Each wave's 32 rows x CW columns at a time through a part of LDS of its
  // own, a row's 16-byte pieces exchanged by an exclusive or with its number.  Lane l holds row l % 32 and, in element e of tile j, column 32 j + 8
  // (e / 4) + 4 (l / 32) + e % 4.
  constexpr int kSize = OUT == kOutF32 ? 4 : 2;
  constexpr int kFit = S::kSlotBytes / (S::NW * 32 * 32 * kSize);
  constexpr int CT = kFit < TN ? kFit : TN;                   // tiles of columns at a time
  constexpr int CW = CT * 32, kStride = CW * kSize, kPieces = kStride / 16;
  static_assert(CT > 0 && TN % CT == 0, "the pieces fit one slot");
  uint8_t* const mine = s0 + wave * 32 * kStride;
  const bool whole = reinterpret_cast<uintptr_t>(out) % 16 == 0 && (ldo * kSize) % 16 == 0 &&
                     (n * kSize) % 16 == 0;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int64_t row0 = m0 + arow + i * 32;
#pragma unroll
    for (int j0 = 0; j0 < TN; j0 += CT) {
      const int64_t col0 = n0 + brow + j0 * 32;
#pragma unroll
      for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16& c = acc[i][j0 + j];
          const int byte = (j * 32 + 8 * g + 4 * h) * kSize;
          uint8_t* p = mine + r * kStride + ((byte / 16) ^ (r & (kPieces - 1))) * 16 + byte % 16;
          if constexpr (OUT == kOutF32)
            *reinterpret_cast<f32x4*>(p) = f32x4{c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]};
          else
            *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(c[4 * g], c[4 * g + 1]),
                                                      bf16_pair(c[4 * g + 2], c[4 * g + 3]));
        }
      __builtin_amdgcn_wave_barrier();
      if (whole) {
#pragma unroll
        for (int it = 0; it < kPieces / 2; ++it) {
          const int q = it * 64 + lane, row = q / kPieces, cb16 = q % kPieces;
          const u32x4 v = *reinterpret_cast<const u32x4*>(mine + row * kStride +
                                                            (cb16 ^ (row & (kPieces - 1))) * 16);
          const int64_t col = col0 + cb16 * (16 / kSize);
          if (row0 + row < m && col < n)
            __builtin_nontemporal_store(
                v, reinterpret_cast<u32x4*>(static_cast<uint8_t*>(out) +
                                            ((row0 + row) * ldo + col) * kSize));
        }
      } else {
        for (int q = lane; q < 32 * CW; q += 64) {
          const int row = q / CW;
          const int64_t col = col0 + q % CW;
          if (row0 + row < m && col < n) {
            const int byte = (q % CW) * kSize;
            const uint8_t* p = mine + row * kStride + ((byte / 16) ^ (row & (kPieces - 1))) * 16 +
                               byte % 16;
            if constexpr (OUT == kOutF32)
              static_cast<float*>(out)[(row0 + row) * ldo + col] = *reinterpret_cast<const float*>(p);
            else
              static_cast<unsigned short*>(out)[(row0 + row) * ldo + col] =
                  *reinterpret_cast<const unsigned short*>(p);
          }
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

template <int WM, int WN, int TM, int TN, bool RAGGED>
hipError_t launch_tiled(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m,
                        const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k,
                        void* out, int out_dtype, int64_t ldo, hipStream_t stream) {
  using S = TileShape<WM, WN, TM, TN, RAGGED>;
  const int64_t tm = (m + S::BM - 1) / S::BM, tn = (n + S::BN - 1) / S::BN;
  if (tm > ((int64_t(1) << 32) - 1) / (S::NW * 64) / tn) return hipErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(tm * tn);
  if (out_dtype == kOutF32)
    mxfp4_gemm_tiled<WM, WN, TM, TN, RAGGED, 0><<<grid, S::NW * 64, 0, stream>>>(
        a_codes, a_scales, m, b_codes, b_scales, n, k, out, ldo, static_cast<int>(tm),
        static_cast<int>(tn));
  else
    mxfp4_gemm_tiled<WM, WN, TM, TN, RAGGED, 1><<<grid, S::NW * 64, 0, stream>>>(
        a_codes, a_scales, m, b_codes, b_scales, n, k, out, ldo, static_cast<int>(tm),
        static_cast<int>(tn));
  return hipGetLastError();
}

template <int NW, int SF, int LF, bool RAGGED, bool S_IS_B>
hipError_t launch_stream(const uint8_t* s_codes, const uint8_t* s_scales, int64_t s_rows,
                         const uint8_t* l_codes, const uint8_t* l_scales, int64_t l_rows,
                         int64_t k, void* out, int out_dtype, int64_t ldo, hipStream_t stream) {
  const int64_t groups = (s_rows + SF * 16 - 1) / (SF * 16);
  if (groups > 0x7FFFFF) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(groups), static_cast<unsigned>((l_rows + LF * 16 - 1) / (LF * 16)));
  if (out_dtype == kOutF32)
    mxfp4_gemm_stream<NW, SF, LF, RAGGED, S_IS_B, 0><<<grid, NW * 64, 0, stream>>>(
        s_codes, s_scales, s_rows, l_codes, l_scales, l_rows, k, out, ldo);
  else
    mxfp4_gemm_stream<NW, SF, LF, RAGGED, S_IS_B, 1><<<grid, NW * 64, 0, stream>>>(
        s_codes, s_scales, s_rows, l_codes, l_scales, l_rows, k, out, ldo);
  return hipGetLastError();
}

template <int LF, bool RAGGED, bool S_IS_B>
hipError_t stream_of(const Mxfp4Plan& p, const uint8_t* sc, const uint8_t* ss, int64_t s_rows,
                     const uint8_t* lc, const uint8_t* ls, int64_t l_rows, int64_t k, void* out,
                     int dt, int64_t ldo, hipStream_t st) {
  if (p.waves == 4)
    return launch_stream<4, 2, LF, RAGGED, S_IS_B>(sc, ss, s_rows, lc, ls, l_rows, k, out, dt, ldo, st);
  if (p.sf == 1)
    return launch_stream<8, 1, LF, RAGGED, S_IS_B>(sc, ss, s_rows, lc, ls, l_rows, k, out, dt, ldo, st);
  if constexpr (LF <= 2)
    if (p.sf == 3)
      return launch_stream<8, 3, LF, RAGGED, S_IS_B>(sc, ss, s_rows, lc, ls, l_rows, k, out, dt, ldo, st);
  if constexpr (LF == 1)
    if (p.sf == 4)
      return launch_stream<8, 4, LF, RAGGED, S_IS_B>(sc, ss, s_rows, lc, ls, l_rows, k, out, dt, ldo, st);
  return launch_stream<8, 2, LF, RAGGED, S_IS_B>(sc, ss, s_rows, lc, ls, l_rows, k, out, dt, ldo, st);
}

template <bool RAGGED>
hipError_t gemm_of(const Mxfp4Plan& p, const uint8_t* ac, const uint8_t* as, int64_t m,
                   const uint8_t* bc, const uint8_t* bs, int64_t n, int64_t k, void* out, int dt,
                   int64_t ldo, hipStream_t st) {
  if (p.tile == 256)
    return launch_tiled<2, 4, 4, 2, RAGGED>(ac, as, m, bc, bs, n, k, out, dt, ldo, st);
  if (p.tile == 128)
    return launch_tiled<2, 2, 2, 2, RAGGED>(ac, as, m, bc, bs, n, k, out, dt, ldo, st);
  if (p.s_is_b) {
    if (p.lf == 1) return stream_of<1, RAGGED, true>(p, bc, bs, n, ac, as, m, k, out, dt, ldo, st);
    if (p.lf == 2) return stream_of<2, RAGGED, true>(p, bc, bs, n, ac, as, m, k, out, dt, ldo, st);
    return stream_of<4, RAGGED, true>(p, bc, bs, n, ac, as, m, k, out, dt, ldo, st);
  }
  if (p.lf == 1) return stream_of<1, RAGGED, false>(p, ac, as, m, bc, bs, n, k, out, dt, ldo, st);
  if (p.lf == 2) return stream_of<2, RAGGED, false>(p, ac, as, m, bc, bs, n, k, out, dt, ldo, st);
  return stream_of<4, RAGGED, false>(p, ac, as, m, bc, bs, n, k, out, dt, ldo, st);
}

}  // namespace

hipError_t launch_mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m,
                             const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k,
                             void* out, int out_dtype, int64_t ldo, hipStream_t stream) {
  const Mxfp4Plan p = mxfp4_plan(m, n, k);
  return p.ragged ? gemm_of<true>(p, a_codes, a_scales, m, b_codes, b_scales, n, k, out, out_dtype,
                                  ldo, stream)
                  : gemm_of<false>(p, a_codes, a_scales, m, b_codes, b_scales, n, k, out, out_dtype,
                                   ldo, stream);
}

}  // namespace nvfp4
