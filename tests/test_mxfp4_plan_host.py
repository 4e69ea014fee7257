"""The rule that picks mxfp4_gemm's kernel, on the CPU: csrc/mxfp4_plan.h compiled
for the host.  Each shape of the GPU tests has the kernel that it is for, and every
kernel has one."""
import os
import subprocess

import pytest

from conftest import ROOT
import test_gpu_mxfp4_kernels as kernels

CSRC = os.path.join(ROOT, "nvfp4_w4a4_quantized_03_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "mxfp4_plan.h"
int main() {
  long long m, n, k;
  while (std::scanf("%lld %lld %lld", &m, &n, &k) == 3) {
    const nvfp4::Mxfp4Plan p = nvfp4::mxfp4_plan(m, n, k);
    std::printf("%d %d %d %d %d %d\n", p.tile, p.waves, p.sf, p.lf, p.ragged, p.s_is_b);
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """Plans of shapes: [(tile, waves, sf, lf, ragged, s_is_b)]."""
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(PROGRAM)
    built = subprocess.run(["g++", "-std=c++17", "-O1", "-I" + CSRC, str(at / "plan.cpp"), "-o",
                            str(at / "plan")], capture_output=True, text=True)
    assert built.returncode == 0, built.stderr

    def of(shapes):
        ran = subprocess.run([str(at / "plan")], input="\n".join("%d %d %d" % s for s in shapes),
                             capture_output=True, text=True, timeout=20)
        assert ran.returncode == 0
        return [tuple(int(x) for x in line.split()) for line in ran.stdout.splitlines()]
    return of


def test_shapes_reach_the_kernels_they_are_for(plans):
    shapes = [s for s, _ in kernels.KERNELS]
    for (shape, want), got in zip(kernels.KERNELS, plans(shapes)):
        assert (got[0] or got[1:4]) == want, (shape, got)
        assert got[4] == (shape[2] % 128 != 0), (shape, got)
        if not got[0]:
            assert got[5] == (shape[0] <= shape[1]), (shape, got)


def test_every_kernel_has_a_shape(plans):
    got = set(p if p[0] == 0 else p[:5] for p in plans([s for s, _ in kernels.KERNELS]))
    want = {(tile, 0, 0, 0, ragged) for tile in (256, 128) for ragged in (0, 1)}
    for lf, most in ((1, 4), (2, 3), (4, 2)):
        for waves, sf in [(8, i + 1) for i in range(most)] + [(4, 2)]:
            want |= {(0, waves, sf, lf, ragged, of_b) for ragged in (0, 1) for of_b in (0, 1)}
    assert got == want


def test_other_large_shapes(plans):
    """Shapes that the GPU tests name elsewhere as those of a kernel."""
    assert all(p[0] == 256 for p in plans([(2901, 2899, 800), (2900, 2904, 768), (2901, 2899, 1312),
                                           (2900, 2900, 544), (65537, 40000, 32)]))
    assert all(p[0] == 128 for p in plans([(1003, 2500, 5152), (2500, 1003, 2688), (900, 1500, 1312)]))


def test_no_shape_is_left_out(plans):
    """Every plan names a kernel that there is, over the range of sizes."""
    sizes = [1, 15, 16, 17, 32, 33, 64, 65, 128, 4095, 4097, 8193, 12289, 16385, 65535, 65536,
             70001, 1 << 20, 1 << 26]
    shapes = [(m, n, k) for m in sizes for n in sizes for k in (32, 128, 2048, 2080, 1 << 22)]
    for shape, (tile, waves, sf, lf, ragged, s_is_b) in zip(shapes, plans(shapes)):
        if tile:
            assert tile in (128, 256) and min(shape[:2]) > 64, shape
            continue
        assert (waves, sf, lf) in {(8, 1, 1), (8, 2, 1), (8, 3, 1), (8, 4, 1), (4, 2, 1), (8, 1, 2),
                                   (8, 2, 2), (8, 3, 2), (4, 2, 2), (8, 1, 4), (8, 2, 4), (4, 2, 4)}
        few = shape[0] if s_is_b else shape[1]
        assert few <= 16 * lf or (few > 64 and lf == 4 and shape[2] >= 2048), shape
