"""The cut of decodes' keys into pieces, on the CPU: csrc/kv_cut.h compiled for
the host.  The pieces must cover the keys and stay within the bound that the
launch and the workspace are sized by, over lengths up to the longest that the
calls accept."""
import os
import subprocess

from conftest import ROOT

CSRC = os.path.join(ROOT, "nvfp4_w4a4_quantized_03_amd", "csrc")

PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>
#include "kv_cut.h"
using namespace nvfp4;
static long tried = 0, wrong = 0;

void say(const char* what, size_t n, int most, int kv_heads, long long got, long long bound) {
  if (++wrong <= 10)
    std::printf("wrong: %s, %zu requests of at most %d keys, %d heads: %lld, not %lld\n", what, n, most,
                kv_heads, got, bound);
}

void cut(const std::vector<int>& keys, int kv_heads, int least) {
  // the kernel adds 64 lanes' sums of every 64th length
  float lane[64] = {}, total = 0.0f, most = 0.0f;
  int longest = 0;
  for (size_t i = 0; i < keys.size(); ++i) {
    lane[i & 63] += static_cast<float>(keys[i]);
    if (keys[i] > most) most = static_cast<float>(keys[i]);
    if (keys[i] > longest) longest = keys[i];
  }
  for (float x : lane) total += x;
  const int chunk = piece_keys(total, most, static_cast<float>(keys.size()), kv_heads, least);
  const float per_key = 1.0f / static_cast<float>(chunk);
  int64_t pieces = 0;
  for (int k : keys) {
    const int64_t n = pieces_of(k, chunk, per_key);
    const int64_t want = k < 1 ? 1 : (int64_t(k) + chunk - 1) / chunk;
    if (n != want) say("pieces of a request", keys.size(), k, kv_heads, n, want);
    const int64_t again = chunks_of(k, chunk, 0x7FFFFFFF);
    if (again != want) say("chunks of a request", keys.size(), k, kv_heads, again, want);
    pieces += n;
  }
  ++tried;
  const int64_t bound = pieces_bound(keys.size(), kv_heads);
  if (chunk < least || chunk % 128) say("keys of a piece", keys.size(), longest, kv_heads, chunk, least);
  if (pieces > bound) say("pieces", keys.size(), longest, kv_heads, pieces, bound);
}

int main() {
  std::mt19937_64 rng(7);
  const int mosts[] = {1, 300, 513, 5000, 32768, 131072, 1 << 24, (1 << 24) + 1, 1 << 30,
                       (1 << 30) + 129, 0x7FFFFFFF - 65536};
  const int counts[] = {1, 2, 3, 63, 64, 65, 200, 255, 256, 257, 700, 1023, 1024};
  for (int least : {256, 512})
    for (int kv_heads : {1, 2, 3, 4, 8, 16, 40, 64, 1024, 65536})
      for (int n : counts)
        for (int most : mosts)
          for (int kind = 0; kind < 6; ++kind) {
            std::vector<int> keys(n, most);             // 0: all alike
            for (int i = 0; i < n; ++i) {
              const double u = double(rng() >> 11) / 9007199254740992.0;
              if (kind == 1) keys[i] = int(u * most);
              if (kind == 2) keys[i] = i ? int(u * (most < 700 ? most : 700)) : most;   // one long
              if (kind == 3) keys[i] = i % 4 ? 0 : most;
              if (kind == 4) keys[i] = most / (1 + int(u * 8));
              if (kind == 5) keys[i] = i % 4 ? 1 : most - int(u * (most < 130 ? most : 130));
            }
            cut(keys, kv_heads, least);
          }
  std::printf("%ld tried, %ld wrong\n", tried, wrong);
  return wrong != 0;
}
"""


def test_pieces_cover_and_are_bounded(tmp_path):
    src, exe = tmp_path / "cut.cpp", tmp_path / "cut"
    src.write_text(PROGRAM)
    # -fwrapv: a sum that passes 31 bits wraps as it does on the GPU
    built = subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-ffp-contract=off", "-I" + CSRC,
                            str(src), "-o", str(exe)], capture_output=True, text=True)
    assert built.returncode == 0, built.stderr
    ran = subprocess.run([str(exe)], capture_output=True, text=True, timeout=100)
    assert ran.returncode == 0, ran.stdout
    assert int(ran.stdout.split()[0]) > 1000
