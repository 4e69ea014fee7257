"""MXFP4 (OCP microscaling, 4-bit form), in float64.
TEST INFRASTRUCTURE ONLY (see oracle/__init__.py for the page key).

The pages use NVFP4; this is the 4-bit format with E8M0 scales per 32 elements
that the OCP microscaling specification defines: scale exponent floor(log2
max|x|) less the largest element exponent (2), elements E2M1, rounded to
nearest, ties to the even code, saturating at 6.  Scales are powers of two, so
every quotient below is exact in float64 and every comparison with a midpoint
decides the rounding without error.
"""
import numpy as np

from .formats import E2M1_MAG

BLOCK = 32


def mxfp4_quantize(x):
    """(codes [rows, k/2], scales [rows, k/32]) of finite x [rows, k]."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    b = x.reshape(rows, k // BLOCK, BLOCK)
    top = np.abs(b).max(-1)
    # frexp: top = f 2^e with f in [1/2, 1), so floor(log2 top) = e - 1
    e = np.where(top > 0, np.frexp(top)[1] - 1 - 2, -127)
    e = np.maximum(e, -127)
    a = np.ldexp(np.abs(b), -e[..., None])
    grid = [float(v) for v in E2M1_MAG]
    code = np.zeros(b.shape, dtype=np.uint8)
    for i in range(7):
        mid = 0.5 * (grid[i] + grid[i + 1])
        up = (a > mid) | ((a == mid) & ((i + 1) % 2 == 0))
        code += up.astype(np.uint8)
    code |= np.signbit(b).astype(np.uint8) << 3
    code = code.reshape(rows, k)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).astype(np.uint8)


def mxfp4_values(codes, scales):
    """float64 values [rows, k] of packed codes and scales (0xFF: NaN)."""
    codes = np.asarray(codes)
    c = np.empty((codes.shape[0], 2 * codes.shape[1]), dtype=np.uint8)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    v = np.array([float(g) for g in E2M1_MAG])[c & 7]
    v = np.where(c & 8, -v, v)
    s = np.ldexp(1.0, np.asarray(scales).astype(int) - 127)
    s = np.where(np.asarray(scales) == 255, np.nan, s)
    return v * np.repeat(s, BLOCK, axis=1)
