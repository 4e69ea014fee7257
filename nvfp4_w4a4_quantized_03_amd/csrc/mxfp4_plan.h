// Which kernel takes an MXFP4 product: plain C++, so that a test on the host can
// say which one each of its shapes is for.
#pragma once

#include <stdint.h>

namespace nvfp4 {

// Tiles of 256 x 256 or 128 x 128 (tile), or (tile 0) the streaming kernel:
// workgroups of `waves` waves that share K, 16 sf rows of the streamed operand (B
// where s_is_b, else A) against 16 lf of the other.  ragged: k is no multiple of 128.
struct Mxfp4Plan {
  int tile, waves, sf, lf;
  bool ragged, s_is_b;
};

// Tiles of 256 x 256 (one workgroup a CU) or 128 x 128 (two).  Times of a round
// of 256 CUs at K = 5120, full and partly filled: 42 and 30 us for the large
// tile, 27 and, for at most one workgroup a CU, 16.5 for the small one; the
// sums over a call's rounds choose.  (1003 x 17536 72 us with large, 68 with
// small tiles; 300 x 5120 28 and 17; 1024 x 10240 35 and 44; 4096 x 12288 125
// and 163; 1500 x 12288 69 and 68.  Only the times' ratio counts, which other K, ragged
// rows and float32 outputs keep near enough: 1003 x 17536 at K = 1024 22.6 and 20.0, at
// 5152 to float32 104 and 89; K = 1024: 4096 x 12288 41 and 48, 1024 x 10240 11.0 and
// 13.2.  Large tiles for the whole rounds and small ones for the rest in a second
// launch: 1003 x 17536 6 % longer, 8192 x 8448 2 %, 1500 x 12288 7 % less.)
inline bool large_tiles(int64_t m, int64_t n) {
  const double large = static_cast<double>((m + 255) / 256) * ((n + 255) / 256);
  const double small = static_cast<double>((m + 127) / 128) * ((n + 127) / 128);
  const double fl = __builtin_floor(large / 256), fs = __builtin_floor(small / 512);
  const double rl = large - 256 * fl, rs = small - 512 * fs;
  return 42.0 * fl + (rl > 0 ? 30.0 : 0.0) <=
         27.0 * fs + (rs > 256 ? 27.0 : rs > 0 ? 16.5 : 0.0);
}

// Products whose tiles would leave most CUs idle while each goes through a long K:
// one round of streaming workgroups, of 16 or 32 rows of the longer side against 64
// of the other, whose waves share K.  K = 5120, tiles and streaming: 128 x 128 11.4
// and 9.5 us, 457 x 312 12.1 and 9.7, 128 x 4096 17.8 and 11.9, 700 x 700 22.3 and
// 11.9; 128 x 2048 x 17408 52 and 27.  Shorter K: 512 x 1000 x 2048 7.1 and 6.9, 512
// x 512 x 1024 5.0 and 6.3.
inline int64_t small_groups(int64_t m, int64_t n, int sf) {
  const int64_t s = m <= n ? n : m, l = m <= n ? m : n;
  return (s + 16 * sf - 1) / (16 * sf) * ((l + 63) / 64);
}
inline bool small_product(int64_t m, int64_t n, int64_t k) {
  return k >= 2048 && m < (1 << 16) && n < (1 << 16) && small_groups(m, n, 2) <= 256;
}

// One operand of at most 64 rows.  One round of workgroups of eight waves, one a CU,
// where some SF gives it (the smallest does: 32 x 10240 x 5120 10.7 us with 214
// workgroups of 48 rows, 15.8 with 320 of 32 and 17.5 with 640 of 16; 32 x 5120 x 5120
// 8.3 with 32 rows, 9.9 with 48); otherwise many of four waves with few loads in
// flight, several a CU (32768 x 64 x 5120 39 us against 47 with eight waves, 64 x
// 10240 x 5120 19 against 23).
inline Mxfp4Plan stream_plan(int64_t s_rows, int64_t l_rows, bool ragged, bool s_is_b) {
  const int lf = l_rows <= 16 ? 1 : l_rows <= 32 ? 2 : 4;
  const int most = lf == 1 ? 4 : lf == 2 ? 3 : 2;             // what the registers hold
  const int64_t sf = (s_rows + 16 * 256 - 1) / (16 * 256);
  if (sf <= most) return {0, 8, static_cast<int>(sf), lf, ragged, s_is_b};
  return {0, 4, 2, lf, ragged, s_is_b};
}

inline Mxfp4Plan mxfp4_plan(int64_t m, int64_t n, int64_t k) {
  const bool ragged = k % 128 != 0;
  if (m <= 64 && (n > 64 || m <= n)) return stream_plan(n, m, ragged, true);
  if (n <= 64) return stream_plan(m, n, ragged, false);
  if (small_product(m, n, k))
    return {0, 8, small_groups(m, n, 1) <= 256 ? 1 : 2, 4, ragged, m <= n};
  return {large_tiles(m, n) ? 256 : 128, 0, 0, 0, ragged, false};
}

}  // namespace nvfp4
