"""MXFP4 on the CPU: the oracle against the format's definition, the C ABI's
and the binding's refusals.  Nothing is launched."""
import os

import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_03_amd as nv
import oracle
from test_attention_host import _OnGpu, at, gpu, no_library  # noqa: F401

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(nv.LIB_PATH):
        pytest.fail("library not built: run __graft_entry__.build()")
    return nv.library()


# ------------------------------------------------------------------ oracle

def test_worked_block():
    """One block by hand: the largest is 13, floor(log2 13) = 3, scale 2 (byte
    128); 13/2 = 6.5 saturates, 5 and 3.5 are ties and go to the even codes
    (4 and 4), 0.5 = 0.25 units ties to 0, -0.0 keeps its sign."""
    x = np.zeros((1, 32))
    x[0, :8] = [13.0, -10.0, 7.0, 0.5, 0.50001, -0.0, 3.0, -1.5]
    codes, scales = oracle.mxfp4_quantize(x)
    assert scales.tolist() == [[128]]
    low = [7, 8 | 6, 6, 0, 1, 8, 3, 8 | 2]
    assert codes[0, :4].tolist() == [a | (b << 4) for a, b in zip(low[0::2], low[1::2])]
    assert not codes[0, 4:].any()


def test_scales_are_e8m0():
    """torch's E8M0 decoder agrees with the oracle's scales on every byte."""
    b = torch.arange(255, dtype=torch.uint8)
    want = b.view(torch.float8_e8m0fnu).double().numpy()
    codes = np.full((255, 16), 0x22, dtype=np.uint8)          # 1.0 everywhere
    got = oracle.mxfp4_values(codes, b.numpy()[:, None])
    assert np.array_equal(got, np.repeat(want[:, None], 32, 1))
    assert np.isnan(oracle.mxfp4_values(codes[:1], np.array([[255]]))).all()


@pytest.mark.parametrize("e", [-140, -126, -125, -124, -3, 0, 100, 127])
def test_nearest_by_brute_force(e):
    """Every bf16 mantissa and 40 exponents below the largest: the value is
    the nearest of the grid, ties to the even code."""
    top = min(1.0 * 2.0 ** e * 1.9921875, 3.38953139e38)
    x = [top]
    for d in range(40):
        x += [s * (1 + m / 128) * 2.0 ** (e - d) for m in range(128) for s in (1, -1)]
    x = np.array(x, dtype=np.float64)
    x = x[np.abs(x) <= top]
    for i in range(0, len(x), 31):
        b = np.zeros(32)
        part = x[i:i + 31]
        b[0], b[1:1 + len(part)] = top, part
        codes, scales = oracle.mxfp4_quantize(b[None])
        s = 2.0 ** (int(scales[0, 0]) - 127)
        assert s == 2.0 ** max(np.floor(np.log2(top)) - 2, -127)
        c = np.stack((codes[0] & 15, codes[0] >> 4), 1).ravel()
        for v, code in zip(b, c):
            a = min(abs(v) / s, 6.0)
            off = [abs(a - g) for g in GRID]
            best = min(off)
            near = [j for j, o in enumerate(off) if o == best]
            assert int(code & 7) == next(j for j in near if len(near) == 1 or j % 2 == 0)
            assert bool(code & 8) == bool(np.signbit(v))


def test_values_of_codes():
    codes = np.arange(256, dtype=np.uint8).reshape(16, 16)
    scales = np.arange(120, 136, dtype=np.uint8)[:, None]
    got = oracle.mxfp4_values(codes, scales)
    for r in range(16):
        for j in range(32):
            c = (codes[r, j // 2] >> (4 * (j % 2))) & 15
            c = int(c)
            assert got[r, j] == (-1) ** (c >> 3) * GRID[c & 7] * 2.0 ** (int(scales[r, 0]) - 127)


# ----------------------------------------------------------------- refusals

def quantize(lib, **kw):
    a = dict(x=at(0), dt=1, rows=3, k=64, ldx=64, codes=at(1), scales=at(2))
    a.update(kw)
    return lib.mxfp4_quantize(*a.values(), None)


def test_quantize_validation(lib):
    for kw in ("x", "codes", "scales"):
        assert quantize(lib, **{kw: None}) == INVALID, kw
    for kw in ("rows", "k", "ldx"):
        for v in (0, -32, 1 << 50):
            assert quantize(lib, **{kw: v}) != OK, (kw, v)
    assert quantize(lib, k=48, ldx=48) == INVALID
    assert quantize(lib, ldx=56) == INVALID
    assert quantize(lib, dt=2) == UNSUPPORTED
    assert quantize(lib, dt=7) == UNSUPPORTED
    assert quantize(lib, x=at(0) + 8) == MISALIGNED
    assert quantize(lib, ldx=66) == MISALIGNED
    assert quantize(lib, codes=at(1) + 8) == MISALIGNED
    assert quantize(lib, codes=at(0) + 128) == INVALID
    assert quantize(lib, scales=at(0) + 5) == INVALID
    assert quantize(lib, scales=at(1) + 5) == INVALID


def dequantize(lib, **kw):
    a = dict(codes=at(0), scales=at(1), rows=3, k=64, out=at(2), dt=1, ldo=64)
    a.update(kw)
    return lib.mxfp4_dequantize(*a.values(), None)


def test_dequantize_validation(lib):
    for kw in ("out", "codes", "scales"):
        assert dequantize(lib, **{kw: None}) == INVALID, kw
    for kw in ("rows", "k", "ldo"):
        for v in (0, -32, 1 << 50):
            assert dequantize(lib, **{kw: v}) != OK, (kw, v)
    assert dequantize(lib, k=16) == INVALID
    assert dequantize(lib, dt=2) == UNSUPPORTED
    assert dequantize(lib, out=at(2) + 4) == MISALIGNED
    assert dequantize(lib, ldo=68) == MISALIGNED
    assert dequantize(lib, codes=at(0) + 4) == MISALIGNED
    assert dequantize(lib, out=at(0)) == INVALID
    assert dequantize(lib, out=at(1)) == INVALID


def gemm(lib, **kw):
    a = dict(ac=at(0), asc=at(1), m=5, bc=at(2), bsc=at(3), n=7, k=64, out=at(4), dt=1, ldo=7)
    a.update(kw)
    return lib.mxfp4_gemm(*a.values(), None)


def test_gemm_validation(lib):
    for kw in ("ac", "asc", "bc", "bsc", "out"):
        assert gemm(lib, **{kw: None}) == INVALID, kw
        if kw != "out":
            assert gemm(lib, **{kw: at(5) + 8}) == MISALIGNED, kw
    for kw in ("m", "n", "k", "ldo"):
        for v in (0, -32, 1 << 50):
            assert gemm(lib, **{kw: v}) != OK, (kw, v)
    assert gemm(lib, k=48) == INVALID
    assert gemm(lib, ldo=6) == INVALID
    assert gemm(lib, k=(1 << 22) + 32) == UNSUPPORTED
    assert gemm(lib, dt=2) == UNSUPPORTED
    assert gemm(lib, out=at(4) + 2) == MISALIGNED
    for on in (0, 1, 2, 3):
        assert gemm(lib, out=at(on)) == INVALID, on


def u8(*shape):
    return gpu(*shape, dtype=torch.uint8)


def test_binding_refuses(no_library):  # noqa: F811
    good = nv.MXFP4(u8(4, 32), u8(4, 2))
    bad = [nv.MXFP4(torch.zeros(4, 32, dtype=torch.uint8), u8(4, 2)),
           nv.MXFP4(gpu(4, 32), u8(4, 2)), nv.MXFP4(u8(4, 32), u8(4, 3)),
           nv.MXFP4(u8(4, 32), u8(3, 2)), nv.MXFP4(u8(4, 32), gpu(4, 2)),
           nv.MXFP4(u8(4, 64)[:, ::2], u8(4, 2)), nv.MXFP4(u8(128), u8(8))]
    for q in bad:
        with pytest.raises(ValueError):
            nv.mxfp4_dequantize(q)
        with pytest.raises(ValueError):
            nv.mxfp4_gemm(q, good)
        with pytest.raises(ValueError):
            nv.mxfp4_gemm(good, q)
    for call in (lambda: nv.mxfp4_gemm(good, nv.MXFP4(u8(4, 64), u8(4, 4))),
                 lambda: nv.mxfp4_gemm(good, good, torch.float16),
                 lambda: nv.mxfp4_gemm(good, good, out=gpu(4, 5)),
                 lambda: nv.mxfp4_gemm(good, good, out=gpu(4, 4, dtype=torch.float32)),
                 lambda: nv.mxfp4_dequantize(good, torch.float64),
                 lambda: nv.mxfp4_dequantize(good, out=gpu(4, 65)),
                 lambda: nv.mxfp4_quantize(torch.zeros(4, 64)),
                 lambda: nv.mxfp4_quantize(gpu(4, 64, dtype=torch.float16)),
                 lambda: nv.mxfp4_quantize(gpu(64, 4).t()),
                 lambda: nv.mxfp4_quantize(gpu(4, 64), out=(u8(4, 32), u8(4, 4))),
                 lambda: nv.mxfp4_quantize(gpu(4, 64), out=(u8(4, 32), gpu(4, 2)))):
        with pytest.raises(ValueError):
            call()
