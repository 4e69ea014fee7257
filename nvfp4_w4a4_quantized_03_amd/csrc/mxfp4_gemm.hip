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
// consecutive rows fall on different banks; its four scale bytes are one dword.
// Where k is no multiple of 128 a row's scales begin at any byte: two dwords
// hold them, joined by the row's shift; blocks past k are read as zeros, codes
// and scales (beyond the resource's range, and masked).
//
// The products are computed transposed (B's rows down, A's across), so that a
// lane holds four consecutive columns of one row of Y.  Tiles leave through LDS
// in whole 16-byte pieces.
constexpr int kBK = 128;
constexpr int kRowBytes = kBK / 2;

__device__ __forceinline__ int piece_xor(int row) { return ((row >> 1) ^ (row >> 3)) & 3; }

// One operand's stage loads of a wave: ROWS x 64 bytes of codes, and one dword
// of scales a row (two if RAGGED).  Offsets are 32-bit, from the tile's first
// row; rows past the last read the last.
template <int ROWS, int NW, bool RAGGED>
struct StageLoads {
  static constexpr int kCodes = ROWS / 16 / NW;
  static constexpr int kWords = RAGGED ? 2 : 1;
  static constexpr int kScales = (ROWS * kWords + 64 * NW - 1) / (64 * NW);
  static constexpr int kIssues = kCodes + kScales;
  static constexpr int kScaleBytes = kScales * NW * 256;      // of a slot
  static_assert(ROWS % (16 * NW) == 0, "rows split evenly over the waves");
  __amdgpu_buffer_rsrc_t codes, scales;
  unsigned code_off[kCodes], scale_off[kScales];

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
    for (int i = 0; i < kScales; ++i) {
      const int q = (wave * kScales + i) * 64 + lane, row = q / kWords;
      scale_off[i] = ((static_cast<unsigned>(s0 - s_from) +
                       static_cast<unsigned>(row < last ? row : last) * blocks) & ~3u) +
                     (q % kWords) * 4;
    }
  }

  // `left`: blocks from this stage's first to the end of K (below 4 only in
  // the last stage of a ragged K)
  __device__ __forceinline__ void issue(int stage, int left, uint8_t* lds_codes,
                                        uint8_t* lds_scales, int wave, int lane) const {
#pragma unroll
    for (int i = 0; i < kCodes; ++i) {
      unsigned off = code_off[i];
      if constexpr (RAGGED) {
        const int q = (wave * kCodes + i) * 64 + lane;
        if (((q & 3) ^ piece_xor(q >> 2)) >= left) off = 0x80000000u;
      }
      lds_buf16(codes, lds_codes + (wave * kCodes + i) * 1024, off, stage * kRowBytes);
    }
#pragma unroll
    for (int i = 0; i < kScales; ++i)
      lds_buf4(scales, lds_scales + (wave * kScales + i) * 256, scale_off[i], stage * 4);
  }
};

// A wave's operands of one k-step of T tiles of 32 rows, and the scales of a
// stage (byte 0: the first k-step's block of this half-wave, byte 2: the
// second's).
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

// The scale words of T rows as LDS has them, and what the products take of
// them: byte 0 and byte 2 are this half-wave's blocks of the two k-steps.
// Taken apart so that nothing waits for the read before the products do.
template <int T, bool RAGGED>
struct Scales {
  u32x2 w[T];
  __device__ __forceinline__ void read(const uint8_t* lds, int row) {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if constexpr (RAGGED) w[t] = *reinterpret_cast<const u32x2*>(lds + row * 8 + t * 256);
      else w[t][0] = *reinterpret_cast<const unsigned*>(lds + row * 4 + t * 128);
    }
  }
  __device__ __forceinline__ void take(unsigned (&s)[T], int half, const unsigned (&shift)[T],
                                       unsigned mask) const {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      s[t] = w[t][0];
      if constexpr (RAGGED) s[t] = __builtin_amdgcn_alignbyte(w[t][1], s[t], shift[t]) & mask;
      s[t] >>= half * 8;
    }
  }
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

template <int WM, int WN, int TM, int TN, bool RAGGED>
struct TileShape {
  static constexpr int NW = WM * WN, BM = WM * TM * 32, BN = WN * TN * 32, NS = 4;
  using LoadsA = StageLoads<BM, NW, RAGGED>;
  using LoadsB = StageLoads<BN, NW, RAGGED>;
  static constexpr int kSlotBytes = (BM + BN) * kRowBytes + LoadsA::kScaleBytes + LoadsB::kScaleBytes;
  static constexpr int kIssues = LoadsA::kIssues + LoadsB::kIssues;
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
      s2[S::kSlotBytes], s3[S::kSlotBytes];
  uint8_t* const slots[NS] = {s0, s1, s2, s3};

  // workgroups are dealt to the 8 XCDs in turn: each XCD takes a contiguous
  // range of tiles, in groups of 8 tiles of rows, so that those that run
  // together share panels in its L2
  const int ntiles = tiles_m * tiles_n;
  int bid = blockIdx.x;
  if (ntiles % 8 == 0) bid = (bid % 8) * (ntiles / 8) + bid / 8;
  constexpr int kGroup = 8;
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

  constexpr int kB = S::BM * kRowBytes, kSA = kB + S::BN * kRowBytes,
                kSB = kSA + S::LoadsA::kScaleBytes;
  auto issue = [&](int stage, uint8_t* slot) {
    const int st = stage < nk ? stage : nk - 1;    // past the end: the last again
    const int left = blocks - 4 * st;
    la.issue(st, left, slot, slot + kSA, wave, lane);
    lb.issue(st, left, slot + kB, slot + kSB, wave, lane);
  };
#pragma unroll
  for (int st = 0; st < NS - 1; ++st) issue(st, slots[st]);
  __builtin_amdgcn_s_waitcnt(kVmcntKeepOf((NS - 2) * S::kIssues));
  stage_barrier();

  // places of the lane's first piece (k-step 0; that of k-step 1 is 32 bytes
  // off, exchanged) and first row
  const int h = lane >> 5, r = lane & 31;
  const int lane_at = r * kRowBytes + (h ^ piece_xor(r)) * 16;
  const int a0 = arow * kRowBytes + lane_at, a1 = a0 ^ 32;
  const int b0 = kB + brow * kRowBytes + lane_at, b1 = b0 ^ 32;
  const int ra = arow + r, rb = brow + r;
  Operand<TM> ca, na;
  Operand<TN> cb, nb;
  unsigned sa[TM], sb[TN];
  read_codes(ca, slots[0], a0);
  read_codes(cb, slots[0], b0);
  Scales<TM, RAGGED> ta;
  Scales<TN, RAGGED> tb;
  ta.read(slots[0] + kSA, ra);
  tb.read(slots[0] + kSB, rb);
  ta.take(sa, h, ashift, nk == 1 ? tail_mask : ~0u);
  tb.take(sb, h, bshift, nk == 1 ? tail_mask : ~0u);

  for (int kt0 = 0; kt0 < nk; kt0 += NS) {
#pragma unroll
    for (int u = 0; u < NS; ++u) {
      const int kt = kt0 + u;
      if (kt < nk) {
      uint8_t* const slot = slots[u];
      uint8_t* const next = slots[(u + 1) % NS];
      issue(kt + NS - 1, slots[(u + NS - 1) % NS]);
      read_codes(na, slot, a1);
      read_codes(nb, slot, b1);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = product<0>(cb.code[j], sb[j], ca.code[i], sa[i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(kVmcntKeepOf((NS - 2) * S::kIssues));
      stage_barrier();
      read_codes(ca, next, a0);
      read_codes(cb, next, b0);
      ta.read(next + kSA, ra);
      tb.read(next + kSB, rb);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = product<1>(nb.code[j], sb[j], na.code[i], sa[i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
      const unsigned mask = kt + 2 >= nk ? tail_mask : ~0u;
      ta.take(sa, h, ashift, mask);
      tb.take(sb, h, bshift, mask);
      }
    }
  }
  // no fill may still be writing LDS when it is used again or released
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();

  // Each wave's 32 rows x CW columns at a time through a part of LDS of its
  // own.  Lane l holds row l % 32 and, in element e of tile j, column 32 j + 8
  // (e / 4) + 4 (l / 32) + e % 4.
  constexpr int kSize = OUT == kOutF32 ? 4 : 2;
  constexpr int CT = OUT == kOutF32 && TN > 2 ? 2 : TN;       // tiles of columns at a time
  constexpr int CW = CT * 32, kStride = CW * kSize + 16;
  static_assert(S::NW * 32 * kStride <= S::kSlotBytes, "the pieces fit one slot");
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
          uint8_t* p = mine + r * kStride + (j * 32 + 8 * g + 4 * h) * kSize;
          if constexpr (OUT == kOutF32)
            *reinterpret_cast<f32x4*>(p) = f32x4{c[4 * g], c[4 * g + 1], c[4 * g + 2], c[4 * g + 3]};
          else
            *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(c[4 * g], c[4 * g + 1]),
                                                      bf16_pair(c[4 * g + 2], c[4 * g + 3]));
        }
      __builtin_amdgcn_wave_barrier();
      if (whole) {
        constexpr int kPieces = CW * kSize / 16;              // of a row
#pragma unroll
        for (int it = 0; it < kPieces / 2; ++it) {
          const int q = it * 64 + lane, row = q / kPieces, cb16 = q % kPieces;
          const u32x4 v = *reinterpret_cast<const u32x4*>(mine + row * kStride + cb16 * 16);
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
            const uint8_t* p = mine + row * kStride + (q % CW) * kSize;
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
