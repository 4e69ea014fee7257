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

// ---------------------------------------------------------------------------
// Tiled kernel.
//
// A workgroup of WM x WN waves computes a tile of WM TM 32 rows of A by WN TN
// 32 rows of B, 128 of K a stage.  Stages go from memory straight to a ring of
// NS slots in LDS; a wave reads its operands one k-step (64 of K) ahead of the
// products that use them.  One wait and one barrier a stage, between its two
// k-steps: stage kt + 1 has landed for everybody before its first operands are
// read, and the slot of stage kt - 1, whose last reads came before the barrier
// of that stage, takes stage kt + NS - 1.
//
// A row's 64 bytes of a stage are four 16-byte pieces (the four blocks),
// exchanged by an exclusive or with the row number so that the operand reads of
// consecutive rows fall on different banks.  Its scales are 4 bytes of a line of
// their own, so they come for four stages at once: read stage by stage they made
// as many requests to L2 as the codes did.  Every wave takes the scales of its
// rows to registers at the start of the four stages, which frees their place in
// LDS for the next four.  Where k is no multiple of 128 a row's scales begin at
// any byte: five dwords hold them, joined by the row's shift, and blocks past k
// are read as zeros (codes beyond the resource's range, scales masked).
//
// The products are computed transposed (B's rows down, A's across), so that a
// lane holds four consecutive columns of one row of Y.  Tiles leave through LDS
// in whole 16-byte pieces.
constexpr int kBK = 128;
constexpr int kRowBytes = kBK / 2;

__device__ __forceinline__ int piece_xor(int row) { return (row >> 2) & 3; }

// One operand's loads of a wave: ROWS x 64 bytes of codes a stage, and 16 bytes
// of scales a row every four stages (a dword more if RAGGED).  Offsets are
// 32-bit, from the tile's first row; rows past the last read the last.
template <int ROWS, int NW, bool RAGGED>
struct Loads {
  static constexpr int kCodes = ROWS / 16 / NW;
  static constexpr int kPerWave = (ROWS + 64 * NW - 1) / (64 * NW);    // rows / 64 of scales
  static constexpr int kScales = kPerWave * (RAGGED ? 2 : 1);
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
      const int q = (wave * kCodes + i) * 64 + lane, row = q >> 2;
      code_off[i] = static_cast<unsigned>(row < last ? row : last) * kbytes +
                    ((q & 3) ^ piece_xor(row)) * 16;
    }
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      const int row = (wave * kPerWave + i) * 64 + lane;
      scale_off[i] = (static_cast<unsigned>(s0 - s_from) +
                      static_cast<unsigned>(row < last ? row : last) * blocks) & ~3u;
    }
  }

  // `left`: blocks from this stage's first to the end of K (below 4 only in
  // the last stage of a ragged K)
  __device__ __forceinline__ void issue_codes(int stage, int left, uint8_t* lds, int wave,
                                              int lane) const {
#pragma unroll
    for (int i = 0; i < kCodes; ++i) {
      unsigned off = code_off[i];
      if constexpr (RAGGED) {
        const int q = (wave * kCodes + i) * 64 + lane;
        if (((q & 3) ^ piece_xor(q >> 2)) >= left) off = 0x80000000u;
      }
      lds_buf16(codes, lds + (wave * kCodes + i) * 1024, off, stage * kRowBytes);
    }
  }

  // the scales of stages 4 window .. 4 window + 3
  __device__ __forceinline__ void issue_scales(int window, uint8_t* lds, int wave) const {
#pragma unroll
    for (int i = 0; i < kPerWave; ++i) {
      lds_buf16(scales, lds + (wave * kPerWave + i) * 1024, scale_off[i], window * 16);
      if constexpr (RAGGED)
        lds_buf4(scales, lds + kRows * 16 + (wave * kPerWave + i) * 256, scale_off[i] + 16,
                 window * 16);
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

// The scales of four stages of T tiles of rows, and of them those of one stage
// as the products take them: byte 0 and byte 2 are this half-wave's blocks of
// the two k-steps.
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
        s[t] = __builtin_amdgcn_alignbyte(U == 3 ? more[t] : w[t][(U + 1) & 3], s[t], shift[t]) & mask;
      s[t] >>= half * 8;
    }
  }
};

template <int I>
struct Index {
  static constexpr int value = I;
};

template <int STEP>
__device__ __forceinline__ f32x16 product(u32x4 a, unsigned sa, u32x4 b, unsigned sb, f32x16 c) {
  const i32x8 x = {static_cast<int>(a[0]), static_cast<int>(a[1]), static_cast<int>(a[2]),
                   static_cast<int>(a[3]), 0, 0, 0, 0};
  const i32x8 y = {static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]),
                   static_cast<int>(b[3]), 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 2 * STEP,
                                                         static_cast<int>(sa), 2 * STEP,
                                                         static_cast<int>(sb));
}

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
  static constexpr int NW = WM * WN, BM = WM * TM * 32, BN = WN * TN * 32, NS = 4;
  using LoadsA = Loads<BM, NW, RAGGED>;
  using LoadsB = Loads<BN, NW, RAGGED>;
  static constexpr int kSlotBytes = (BM + BN) * kRowBytes;
  static constexpr int kScaleBytes = LoadsA::kScaleBytes + LoadsB::kScaleBytes;
  static constexpr int kCodes = LoadsA::kCodes + LoadsB::kCodes;      // loads of a wave
  static constexpr int kScales = LoadsA::kScales + LoadsB::kScales;
};

template <int WM, int WN, int TM, int TN, bool RAGGED, int OUT>
__global__ void __launch_bounds__(WM * WN * 64, 1)
mxfp4_gemm_tiled(const uint8_t* __restrict__ a_codes, const uint8_t* __restrict__ a_scales,
                 int64_t m, const uint8_t* __restrict__ b_codes,
                 const uint8_t* __restrict__ b_scales, int64_t n, int64_t k,
                 void* __restrict__ out, int64_t ldo, int tiles_m, int tiles_n) {
  using S = TileShape<WM, WN, TM, TN, RAGGED>;
  constexpr int NS = S::NS;
  // an object of its own for each slot: a fill of one slot then does not look
  // like a write to what the reads of another wait for
  __shared__ __attribute__((aligned(1024))) uint8_t s0[S::kSlotBytes], s1[S::kSlotBytes],
      s2[S::kSlotBytes], s3[S::kSlotBytes], scale_lds[S::kScaleBytes];

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
  const int blocks = static_cast<int>(k / 32), nk = (blocks + 3) >> 2;

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
  const unsigned tail_mask = (blocks & 3) ? (1u << (8 * (blocks & 3))) - 1u : ~0u;

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  constexpr int kB = S::BM * kRowBytes, kSB = S::LoadsA::kScaleBytes;
  // past the end: the last stage again
  auto issue_a = [&](int stage, uint8_t* slot) {
    const int st = stage < nk ? stage : nk - 1;
    la.issue_codes(st, blocks - 4 * st, slot, wave, lane);
  };
  auto issue_b = [&](int stage, uint8_t* slot) {
    const int st = stage < nk ? stage : nk - 1;
    lb.issue_codes(st, blocks - 4 * st, slot + kB, wave, lane);
  };
  auto issue_scales = [&](int window) {
    la.issue_scales(window, scale_lds, wave);
    lb.issue_scales(window, scale_lds + kSB, wave);
  };
  issue_scales(0);
  issue_a(0, s0);
  issue_b(0, s0);
  issue_a(1, s1);
  issue_b(1, s1);
  issue_a(2, s2);
  issue_b(2, s2);
  __builtin_amdgcn_s_waitcnt(kVmcntKeepOf((NS - 2) * S::kCodes));
  stage_barrier();

  // places of the lane's first piece (k-step 0; that of k-step 1 is 32 bytes
  // off, exchanged) and first row
  const int h = lane >> 5, r = lane & 31;
  const int lane_at = r * kRowBytes + (h ^ piece_xor(r)) * 16;
  const int a0 = arow * kRowBytes + lane_at, a1 = a0 ^ 32;
  const int b0 = kB + brow * kRowBytes + lane_at, b1 = b0 ^ 32;
  Operand<TM> ca, na;
  Operand<TN> cb, nb;
  Scales<TM, RAGGED, S::LoadsA::kRows> wa;
  Scales<TN, RAGGED, S::LoadsB::kRows> wb;
  read_codes(ca, s0, a0);
  read_codes(cb, s0, b0);
  wa.read(scale_lds, arow + r);
  wb.read(scale_lds + kSB, brow + r);

  auto stage = [&](auto index, int kt, uint8_t* slot, uint8_t* next, uint8_t* fill) {
    constexpr int U = decltype(index)::value;
    // The scales of the next four stages go to the place that every wave has
    // read before the barrier of the stage before this one.
    if constexpr (U == 1) issue_scales((kt >> 2) + 1);
    issue_a(kt + NS - 1, fill);
    const unsigned mask = kt + 1 >= nk ? tail_mask : ~0u;
    unsigned sa[TM], sb[TN];
    wa.template take<U>(sa, h, ashift, mask);
    wb.template take<U>(sb, h, bshift, mask);
    read_codes(na, slot, a1);
    read_codes(nb, slot, b1);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = product<0>(cb.code[j], sb[j], ca.code[i], sa[i], acc[i][j]);
    interleave<TM * TN, TM + TN, S::LoadsA::kCodes + (U == 1 ? S::kScales : 0)>();
    // this wave's loads of stage kt + 1 (and of its scales) have landed: those
    // of stage kt + 2 and A's of stage kt + 3 may be in flight, with the scales
    // that were issued between them
    __builtin_amdgcn_s_waitcnt(kVmcntKeepOf((NS - 2) * S::kCodes - S::LoadsB::kCodes +
                                            (U == 1 || U == 2 ? S::kScales : 0)));
    stage_barrier();
    issue_b(kt + NS - 1, fill);
    read_codes(ca, next, a0);
    read_codes(cb, next, b0);
    if constexpr (U == 3) {
      wa.read(scale_lds, arow + r);
      wb.read(scale_lds + kSB, brow + r);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[i][j] = product<1>(nb.code[j], sb[j], na.code[i], sa[i], acc[i][j]);
    interleave<TM * TN, TM + TN, S::LoadsB::kCodes>();
  };
  // whole rounds of four stages, then the one to three that are left: with a
  // condition on a stage inside the loop, the compiler waits for loads that may
  // stay in flight where the paths join
  int kt = 0;
  for (; kt + NS <= nk; kt += NS) {
    stage(Index<0>(), kt, s0, s1, s3);
    stage(Index<1>(), kt + 1, s1, s2, s0);
    stage(Index<2>(), kt + 2, s2, s3, s1);
    stage(Index<3>(), kt + 3, s3, s0, s2);
  }
  if (kt < nk) {
    stage(Index<0>(), kt, s0, s1, s3);
    if (kt + 1 < nk) {
      stage(Index<1>(), kt + 1, s1, s2, s0);
      if (kt + 2 < nk) stage(Index<2>(), kt + 2, s2, s3, s1);
    }
  }
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

}  // namespace

hipError_t launch_mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int64_t m,
                             const uint8_t* b_codes, const uint8_t* b_scales, int64_t n, int64_t k,
                             void* out, int out_dtype, int64_t ldo, hipStream_t stream) {
  // 32-bit offsets within a tile
  if (k <= (int64_t(1) << 22) && m > 64 && n > 64) {
    if (k % kBK == 0)
      return launch_tiled<2, 2, 4, 4, false>(a_codes, a_scales, m, b_codes, b_scales, n, k, out,
                                             out_dtype, ldo, stream);
    return launch_tiled<2, 2, 4, 4, true>(a_codes, a_scales, m, b_codes, b_scales, n, k, out,
                                          out_dtype, ldo, stream);
  }
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
