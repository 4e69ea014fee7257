"""MXFP4 on the GPU (through the C ABI) against the float64 oracle: codes,
scales and values bit for bit; products within the rounding of their sums.

Tolerance of a product: the values are small multiples of powers of two, so
products are exact; a sum of k of them in binary32, in any order, is off by at
most k 2^-24 times the sum of their magnitudes (first order; 1.1 times for the
second), bf16 output by 2^-8 of the value more.
"""
import numpy as np
import pytest
import torch

import nvfp4_w4a4_quantized_03_amd as nv
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def _say(*a):
    print("[gpu-mxfp4]", *a, flush=True)


def host(t):
    return t.cpu().numpy()


def check_quantize(x):
    """x: GPU tensor.  Codes, scales and read-back values are the oracle's."""
    q = nv.mxfp4_quantize(x)
    codes, scales = oracle.mxfp4_quantize(x.double().cpu().numpy())
    assert np.array_equal(host(q.scales), scales)
    assert np.array_equal(host(q.codes), codes)
    want = oracle.mxfp4_values(codes, scales)
    for dt in (F32, BF16):
        got = nv.mxfp4_dequantize(q, dt)
        assert got.dtype == dt
        ref = torch.from_numpy(want).to(dt)
        assert torch.equal(got.cpu(), ref)
        assert torch.equal(torch.signbit(got.cpu()), torch.signbit(ref))
    return q


@pytest.mark.parametrize("rows,k", [(1, 32), (3, 64), (5, 5152), (129, 96), (32, 5120),
                                    (1003, 160)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_and_read_back(rows, k, dtype):
    _say("quantize", rows, k, dtype)
    rng = np.random.default_rng(rows * k)
    x = rng.standard_normal((rows, k)) * 2.0 ** rng.integers(-20, 20, (rows, 1))
    x[rng.random((rows, k)) < 0.05] = 0.0
    check_quantize(torch.from_numpy(x).to(dtype).to(DEV))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_quantize_edges(dtype):
    """Ties, saturation, signed zeros, blocks of zeros, the smallest and largest
    values of the type, subnormals."""
    _say("edges", dtype)
    tiny = 2.0 ** -149 if dtype == F32 else 2.0 ** -133
    big = float(torch.finfo(dtype).max)
    units = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9375, 0.2490234375, 0.251953125]
    rows = []
    for e in (-149, -140, -130, -127, -126, -125, -124, -123, -60, 0, 40, 120, 124):
        b = np.zeros(32)
        b[0] = 7.9375
        b[1:13], b[13:25] = units, [-u for u in units]
        b[25] = -0.0
        with np.errstate(over="ignore"):
            rows.append(np.minimum(np.maximum(b * 2.0 ** e, -big), big))
    rows += [np.zeros(32), np.full(32, -0.0), np.full(32, tiny), np.full(32, -big)]
    one = np.zeros(32)
    one[31] = -tiny
    rows.append(one)
    x = torch.from_numpy(np.array(rows)).to(dtype).to(DEV)
    check_quantize(x)
    check_quantize(x.reshape(1, -1))


def test_quantize_marks_what_is_not_finite():
    x = torch.ones(4, 96, device=DEV)
    x[0, 33], x[1, 64], x[2, 95] = float("inf"), float("-inf"), float("nan")
    q = nv.mxfp4_quantize(x)
    s = host(q.scales)
    assert s[0, 1] == s[1, 2] == s[2, 2] == 255
    v = nv.mxfp4_dequantize(q, F32).view(4, 3, 32)
    bad = torch.isnan(v)
    assert bad[0, 1].all() and bad[1, 2].all() and bad[2, 2].all() and int(bad.sum()) == 96


def test_quantize_strided_rows_and_slices():
    """Rows of a wider tensor; slices of one pair of buffers; strided output."""
    rng = np.random.default_rng(3)
    wide = torch.from_numpy(rng.standard_normal((40, 512))).to(BF16).to(DEV)
    x = wide[:, 64:224]
    q = check_quantize(x)
    codes = torch.full((50, 80), 0xEE, dtype=torch.uint8, device=DEV)
    scales = torch.full((50, 5), 0xEE, dtype=torch.uint8, device=DEV)
    nv.mxfp4_quantize(x, out=(codes[5:45], scales[5:45]))
    assert torch.equal(codes[5:45], q.codes) and torch.equal(scales[5:45], q.scales)
    for t in (codes, scales):
        assert bool((t[:5] == 0xEE).all()) and bool((t[45:] == 0xEE).all())
    for dt in (F32, BF16):
        out = torch.full((40, 512), 7.0, dtype=dt, device=DEV)
        nv.mxfp4_dequantize(q, dt, out=out[:, 128:288])
        assert torch.equal(out[:, 128:288], nv.mxfp4_dequantize(q, dt))
        assert bool((out[:, :128] == 7).all()) and bool((out[:, 288:] == 7).all())


def operand(rng, rows, k, spread=4):
    """Random codes with random scales, and their values."""
    codes = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
    scales = rng.integers(127 - spread, 128 + spread, (rows, k // 32)).astype(np.uint8)
    q = nv.MXFP4(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV))
    return q, oracle.mxfp4_values(codes, scales)


def check_gemm(rng, m, n, k, dt, out=None, spread=4):
    a, av = operand(rng, m, k, spread)
    b, bv = operand(rng, n, k, spread)
    y = nv.mxfp4_gemm(a, b, dt, out=out)
    want, reach = av @ bv.T, np.abs(av) @ np.abs(bv).T
    bound = 1.1 * k * 2.0 ** -24 * reach + (2.0 ** -8 * np.abs(want) if dt == BF16 else 0.0)
    off = np.abs(y.double().cpu().numpy() - want)
    worst = np.unravel_index(np.argmax(off - bound), off.shape)
    assert (off <= bound).all(), (m, n, k, worst, off[worst], bound[worst], want[worst])
    return a, b, y


GEMMS = [(1, 1, 32), (1, 5, 64), (2, 3, 96), (7, 33, 160), (16, 16, 128), (17, 31, 256),
         (32, 64, 512), (33, 65, 288), (64, 100, 1024), (65, 64, 416), (100, 1, 768),
         (1, 300, 2560), (3, 257, 5120), (129, 130, 384), (128, 256, 256), (255, 257, 512),
         (256, 256, 1280), (257, 255, 1056), (300, 520, 2048), (513, 300, 5152)]


# one operand of few rows against each number of rows that a workgroup takes,
# both ways round, one and several rounds of loads
STREAMS = [(1, 4097, 96), (9, 8200, 128), (16, 13000, 160), (3, 16500, 64), (20, 4100, 256),
           (31, 9000, 288), (32, 12400, 128), (50, 5000, 1024), (64, 9000, 96), (5, 100, 9216),
           (40, 33, 12320), (4100, 7, 224), (13000, 32, 128), (9001, 64, 160), (70, 17, 640)]


# small products of a long K, in groups of 64 rows of the shorter side, both ways
# round; and their neighbours in tiles
SMALL = [(457, 312, 2048), (312, 457, 2080), (65, 65, 5152), (65, 4096, 2048), (4090, 66, 2592),
         (700, 700, 2048), (129, 1300, 4128), (128, 128, 2016), (4097, 130, 2048)]


@pytest.mark.parametrize("m,n,k", GEMMS + STREAMS + SMALL)
@pytest.mark.parametrize("dt", [F32, BF16])
def test_gemm(m, n, k, dt):
    _say("gemm", m, n, k, dt)
    check_gemm(np.random.default_rng(m * 7 + n * 3 + k), m, n, k, dt)


def test_gemm_each_block_has_its_scale():
    """One block of one row at a time: the scales of A and of B reach the
    products of their own block and row only."""
    m, n, k = 70, 72, 640
    for r in range(0, 70, 23):
        for blk in range(0, 20, 3):
            codes = np.zeros((m, k // 2), dtype=np.uint8)
            codes[r, blk * 16:blk * 16 + 16] = 0x22                 # 1.0
            sa = np.full((m, k // 32), 130, dtype=np.uint8)
            sa[r, blk] = 124
            bcodes = np.full((n, k // 2), 0x22, dtype=np.uint8)
            sb = np.random.default_rng(blk).integers(120, 134, (n, k // 32)).astype(np.uint8)
            t = [torch.from_numpy(x).to(DEV) for x in (codes, sa, bcodes, sb)]
            y = host(nv.mxfp4_gemm(nv.MXFP4(*t[:2]), nv.MXFP4(*t[2:]), F32))
            want = np.zeros((m, n))
            want[r] = 32 * 2.0 ** -3 * 2.0 ** (sb[:, blk].astype(int) - 127.0)
            assert np.array_equal(y, want), (r, blk)


def test_gemm_scale_range():
    """Scales over the whole range whose sums binary32 holds."""
    _say("scale range")
    rng = np.random.default_rng(9)
    for m, n, k in ((40, 48, 512), (256, 256, 512)):
        a, av = operand(rng, m, k, 1)
        for shift in (-60, 0, 60):
            sb = rng.integers(125 + shift, 129 + shift, (n, k // 32)).astype(np.uint8)
            bc = rng.integers(0, 256, (n, k // 2), dtype=np.uint8)
            y = nv.mxfp4_gemm(a, nv.MXFP4(torch.from_numpy(bc).to(DEV),
                                          torch.from_numpy(sb).to(DEV)), F32)
            bv = oracle.mxfp4_values(bc, sb)
            off = np.abs(y.double().cpu().numpy() - av @ bv.T)
            assert (off <= 1.1 * k * 2.0 ** -24 * (np.abs(av) @ np.abs(bv).T)).all()


@pytest.mark.parametrize("m,n,k", [(5, 40, 96), (20, 300, 512), (300, 300, 512)])
def test_gemm_nan_scales(m, n, k):
    """A row with a NaN scale gives NaN and no other row does."""
    rng = np.random.default_rng(k)
    a, _ = operand(rng, m, k)
    b, _ = operand(rng, n, k)
    a.scales[m // 2, 1] = 255
    b.scales[n - 1, 0] = 255
    y = nv.mxfp4_gemm(a, b, F32).cpu()
    bad = torch.zeros(m, n, dtype=torch.bool)
    bad[m // 2], bad[:, n - 1] = True, True
    assert torch.equal(torch.isnan(y), bad)


@pytest.mark.parametrize("m,n,k", [(3, 70, 96), (30, 130, 256), (260, 270, 512)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_gemm_strided_output(m, n, k, dt):
    """A column range of a wider output, at an odd offset; the rest stays."""
    wide = torch.full((m, n + 39), 5.0, dtype=dt, device=DEV)
    at = 2 if dt == BF16 else 1
    check_gemm(np.random.default_rng(m), m, n, k, dt, out=wide[:, at:at + n])
    assert bool((wide[:, :at] == 5).all()) and bool((wide[:, at + n:] == 5).all())


@pytest.mark.parametrize("m,n,k", [(1, 512, 1024), (32, 1000, 512), (300, 512, 512)])
def test_gemm_repeats_bit_for_bit(m, n, k):
    a, b, y = check_gemm(np.random.default_rng(m), m, n, k, F32)
    for _ in range(3):
        assert torch.equal(nv.mxfp4_gemm(a, b, F32), y)
