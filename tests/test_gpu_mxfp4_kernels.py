"""Each kernel that mxfp4_gemm has, at shapes that its rule gives to it.

The rule is csrc/mxfp4_plan.h; test_mxfp4_plan_host.py holds every shape here to the
kernel that stands beside it, so a changed rule takes no kernel out of the tests.

Products are exact: with scales of 1/2 and 1 (and 2 where K allows it) the values are
multiples of 1/4, products of 1/16, and every partial sum is below 2^20, so binary32
holds each of them, in any order, and outputs have to be equal (BF16: the exact sum
rounded once).
"""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_03_amd as nv
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16

# Shape and kernel: tile 256 or 128, or (waves, 16ths of the streamed operand's rows,
# of the other's).
# Tiles of 256 x 256: odd and even numbers of stages of 256 of K, one to eleven of them
# (scales come for two at once), whole and ragged K, partial tiles on both sides.
LARGE = [(2901, 2899, k) for k in (32, 96, 128, 256, 288, 512, 768, 1024, 1056, 1280, 1312, 2592)] + \
    [(4097, 5000, 640), (1030, 12290, 416), (12290, 1030, 384), (4096, 4096, 256),
     (8192, 2048, 2080)]
# Tiles of 128 x 128 at a long ragged and a long whole K
SMALL_TILES = [(1003, 2500, 5152), (2500, 1003, 5120), (129, 8300, 2592), (1100, 1100, 2688)]
# Few rows of one operand against each choice of rows of the streamed one
FEW = {1: 13, 2: 29, 4: 50}
MANY = {1: {(8, 1): 4001, (8, 2): 8100, (8, 3): 12211, (8, 4): 16300, (4, 2): 16500},
        2: {(8, 1): 4001, (8, 2): 8100, (8, 3): 12211, (4, 2): 12400},
        4: {(8, 1): 4001, (8, 2): 8100, (4, 2): 8300}}


def _stream():
    for lf, rows in FEW.items():
        for (waves, sf), many in MANY[lf].items():
            for k in (640, 672):
                yield (rows, many, k), (waves, sf, lf)
                yield (many, rows, k), (waves, sf, lf)
    # more than one round of loads a wave
    for k in (2208, 2688):
        for lf, rows in FEW.items():
            yield (rows, MANY[lf][4, 2], k), (4, 2, lf)
            yield (MANY[lf][4, 2], rows, k), (4, 2, lf)
    # the same, and small products in groups of 64 rows
    for k in (9344, 9312):
        yield (7, 70, k), (8, 1, 1)
        yield (70, 50, k), (8, 1, 4)
        yield (30, 4100, k), (8, 2, 2)
        yield (300, 130, k), (8, 1, 4)
        yield (130, 2700, k), (8, 2, 4)
        yield (2700, 130, k), (8, 2, 4)


KERNELS = [(s, 256) for s in LARGE] + [(s, 128) for s in SMALL_TILES] + list(_stream())


def _say(*a):
    print("[gpu-mxfp4-kernels]", *a, flush=True)


def operand(rng, rows, k, top):
    codes = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
    scales = rng.integers(126, top, (rows, k // 32)).astype(np.uint8)
    return codes, scales


def on_gpu(x):
    return nv.MXFP4(*(torch.from_numpy(t).to(DEV) for t in x))


def values(x):
    return torch.from_numpy(oracle.mxfp4_values(*x)).float()


def case(m, n, k):
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    # 36 times a product of scales, k of them: below 2^20
    top = 129 if 36 * 4 * k < 2 ** 20 else 128
    assert 36 * k * 4 ** (top - 128) < 2 ** 20
    a, b = operand(rng, m, k, top), operand(rng, n, k, top)
    return on_gpu(a), on_gpu(b), values(a) @ values(b).t()


@pytest.mark.parametrize("m,n,k", [s for s, _ in KERNELS])
def test_products_are_exact(m, n, k):
    _say("exact", m, n, k)
    a, b, want = case(m, n, k)
    for dt in (F32, BF16):
        y = nv.mxfp4_gemm(a, b, dt)
        assert torch.equal(y.cpu(), want.to(dt)), dt
        assert torch.equal(nv.mxfp4_gemm(a, b, dt), y), dt


@pytest.mark.parametrize("m,n,k", [(2901, 2899, 800), (2900, 2904, 768)])
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("at", [0, 2, 8])
def test_large_tiles_in_a_wider_output(m, n, k, dt, at):
    """Columns of a wider output, in whole 16-byte pieces and not; the rest stays."""
    _say("wide", m, n, k, dt, at)
    a, b, want = case(m, n, k)
    wide = torch.full((m + 1, (n + 39) // 8 * 8), 5.0, dtype=dt, device=DEV)
    nv.mxfp4_gemm(a, b, dt, out=wide[:m, at:at + n])
    assert torch.equal(wide[:m, at:at + n].cpu(), want.to(dt))
    wide[:m, at:at + n] = 5.0
    assert bool((wide == 5).all())


@pytest.mark.parametrize("m,n,k", [(2901, 2899, 1312), (2901, 2899, 768), (1003, 2500, 5152),
                                   (2500, 1003, 2688)])
def test_nan_scales_stay_in_their_rows(m, n, k):
    """NaN scales in a first, a middle and a last block; of a last block the next bytes
    in memory are the next row's first."""
    _say("nan", m, n, k)
    a, b, want = case(m, n, k)
    blocks = k // 32
    for r, blk in ((0, 0), (m // 2, blocks // 2), (m - 2, blocks - 1), (m // 3, blocks - 1)):
        a.scales[r, blk] = 255
        want[r] = float("nan")
    for c, blk in ((5, blocks - 1), (n // 2, 1), (n - 1, 0)):
        b.scales[c, blk] = 255
        want[:, c] = float("nan")
    y = nv.mxfp4_gemm(a, b, F32).cpu()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    good = ~torch.isnan(want)
    assert torch.equal(y[good], want[good])


@pytest.mark.parametrize("m,n", [(2901, 2899), (900, 1500)])
def test_each_block_has_its_scale(m, n):
    """One block of some rows at a time, every scale of B another's neighbour differs
    from: the scales reach the products of their own block and row only."""
    _say("blocks", m, n)
    k = 1312
    rng = np.random.default_rng(m)
    sb = rng.integers(120, 134, (n, k // 32)).astype(np.uint8)
    b = on_gpu((np.full((n, k // 2), 0x22, dtype=np.uint8), sb))          # 1.0
    for blk in range(0, 41, 4):
        codes = np.zeros((m, k // 2), dtype=np.uint8)
        sa = rng.integers(120, 134, (m, k // 32)).astype(np.uint8)
        codes[::3, blk * 16:blk * 16 + 16] = 0x22
        y = nv.mxfp4_gemm(on_gpu((codes, sa)), b, F32).cpu().numpy()
        want = np.zeros((m, n))
        want[::3] = 32 * np.exp2(sa[::3, blk, None].astype(float) - 127) * \
            np.exp2(sb[:, blk].astype(float) - 127)
        assert np.array_equal(y, want), blk


def test_scales_over_the_whole_range_in_large_tiles():
    """Scales whose products run from 2^-120 to 2^100, one power a row of B."""
    _say("range")
    m = n = 2900
    k = 544
    a, b, want = case(m, n, k)
    shift = torch.arange(n) % 221 - 120
    b.scales.copy_((b.scales.cpu().int() + shift[:, None].clamp(-120, 100)).to(torch.uint8))
    got = nv.mxfp4_gemm(a, b, F32).cpu().double()
    assert torch.equal(got, want.double() * torch.exp2(shift.double()))
