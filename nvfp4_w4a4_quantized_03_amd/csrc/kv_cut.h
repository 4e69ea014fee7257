// How the keys of requests of few rows (decodes) are cut into pieces: the
// arithmetic that the kernels and the host's sizes have to agree on, as plain
// C++ that host and device compile alike.
#pragma once

#include <stdint.h>

namespace nvfp4 {

constexpr int kFewSlots = 512;         // workgroups that are resident together
constexpr int kMostUneven = 4;

// Keys of a piece, from the requests' `total` and largest `most` keys: one
// piece of the average work for each of kFewSlots workgroups when all are
// alike, down to a quarter of it when they differ; whole tiles of four waves
// (128 keys), at least `least`.  It is more than total * kv_heads / (kFewSlots
// * kMostUneven), so that the pieces are at most pieces_bound.
constexpr int piece_keys(float total, float most, float n, int kv_heads, int least) {
  const float even = n * most / (total > 1.0f ? total : 1.0f);
  const float uneven = even < 1.0f ? 1.0f : even > kMostUneven ? kMostUneven : even;
  const float want = total * static_cast<float>(kv_heads) / (kFewSlots * uneven);
  // capped at as many keys as a request can have
  const int keys = (static_cast<int>(want < 0x7FFF0000p0f ? want : 0x7FFF0000p0f) + 128) & -128;
  return keys > least ? keys : least;
}

// Pieces of a request, at least one: ceil(keys / chunk), the quotient in
// binary32 put right.
constexpr int pieces_of(int keys, int chunk, float per_key) {
  if (keys <= chunk) return 1;
  int count = static_cast<int>(static_cast<float>(keys) * per_key);
  while (static_cast<int64_t>(count) * chunk < keys) ++count;
  while (static_cast<int64_t>(count - 1) * chunk >= keys) --count;
  return count;
}

// Pieces of all requests at most: a last one each, kMostUneven * kFewSlots
// over the heads, and one for the binary32 of piece_keys.
constexpr int64_t pieces_bound(int64_t n_requests, int64_t kv_heads) {
  return n_requests + (kMostUneven * kFewSlots + kv_heads - 1) / kv_heads + 1;
}

// Chunks that `keys` are cut into, between one and `most`.
constexpr int chunks_of(int keys, int chunk, int most) {
  if (keys < 1) return 1;
  // the sum may pass 31 bits
  const int n = static_cast<int>((static_cast<unsigned>(keys) + chunk - 1u) / chunk);
  return n > most ? most : n;
}

}  // namespace nvfp4
