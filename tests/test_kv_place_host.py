"""The addresses of keys in the attention kernels, on the CPU: csrc/kv_place.h
compiled for the host and compared with the same in 64 bits, up to the
longest contexts and the widest token strides that the calls accept."""
import os
import subprocess

from conftest import ROOT

CSRC = os.path.join(ROOT, "nvfp4_w4a4_quantized_03_amd", "csrc")

# Prints each tried span, share and stride whose byte offsets are not those of
# the nearest visible key, and the number of offsets that were compared.
PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include "kv_place.h"
using namespace nvfp4;
static long compared = 0, wrong = 0;

template <int ROWS>
void share(int lo, int hi, int key, int stride) {
  const int g = group_at<ROWS>(hi, key);
  const ByteBounds b = bytes_seen(rows_seen(lo, hi, g), stride);
  for (int r = 0; r < ROWS; ++r) {
    const int64_t seen = int64_t(g) + r < lo ? lo : int64_t(g) + r > hi - 1 ? hi - 1 : int64_t(g) + r;
    const int64_t want = (seen - g) * stride;
    const int64_t got = byte_of(r * stride, b);
    ++compared;
    // inside the 16-key group, so in the share's own page
    if (got != want || seen / kGroupKeys != g / kGroupKeys) {
      if (++wrong <= 10)
        std::printf("wrong: keys [%d, %d) share of %d at %d row %d stride %d: %lld, not %lld\n", lo,
                    hi, ROWS, key, r, stride, (long long)got, (long long)want);
    }
  }
}

void span(int lo, int hi, int stride) {
  const int start = lo & ~15;
  const int64_t at[] = {0, 8, 16, 24, 128, 1024, 16384, (hi - start) / 2 & ~15,
                        (hi - 1 - start) & ~7, ((hi - 1 - start) & ~7) + 8, hi - start + 64};
  for (int64_t a : at) {
    const int64_t key = start + (a & ~int64_t(7));
    if (key > 0x7FFFFFFF) continue;
    share<8>(lo, hi, int(key), stride);
    if (key % 16 == 0) share<16>(lo, hi, int(key), stride);
  }
}

int main() {
  const int his[] = {1, 15, 16, 17, 33, 34, 40, 75, 100, 4099, 16385, 32768, 131073, 149797, 149798,
                     160000, 200000, 838860, 1048577, 1 << 25, 0x7FFFFFFF - 65536};
  // elements 64 .. 2^25 of 2 bytes, 64 .. 2^26 of 1: the widest accepted are
  // the last multiples of 16 bytes below 2^26
  const int strides[] = {64, 128, 256, 512, 2048, 14336, 16384, 1 << 17, (1 << 24) + 16, (1 << 26) - 16};
  for (int hi : his)
    for (int stride : strides) {
      const int los[] = {0, 1, 15, 16, 17, hi / 3, hi - 4096, hi - 129, hi - 17, hi - 16, hi - 1};
      for (int lo : los)
        if (lo >= 0 && lo < hi) span(lo, hi, stride);
    }
  std::printf("%ld compared, %ld wrong\n", compared, wrong);
  return wrong != 0;
}
"""


def test_offsets_of_keys(tmp_path):
    """Every row's offset is that of the nearest key that may be read, in the
    page that was looked up, also where keys times stride passes 2^31."""
    src, exe = tmp_path / "place.cpp", tmp_path / "place"
    src.write_text(PROGRAM)
    # -fwrapv: a product that passes 31 bits wraps as it does on the GPU
    built = subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-I" + CSRC, str(src), "-o",
                            str(exe)], capture_output=True, text=True)
    assert built.returncode == 0, built.stderr
    ran = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert ran.returncode == 0, ran.stdout
    assert int(ran.stdout.split()[0]) > 10000
