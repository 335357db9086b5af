"""CPU oracle for MXFP4 (OCP Microscaling Formats v1.0: E2M1 codes in blocks of
32 with an E8M0 scale) and for the products by expert.

TEST INFRASTRUCTURE, as w4_oracle: plain NumPy in float64, written from the
definitions and sharing no code with the HIP path.  Every float32 or bfloat16
input and every code value is exact in float64.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(w32: np.ndarray):
    """float32 [N, K] -> (codes 0..15 [N, K], scale bytes [N, K/32])."""
    n, k = w32.shape
    b = w32.astype(np.float64).reshape(n, k // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    e = np.where(amax > 0, np.frexp(amax)[1] - 1 - 2, -127)  # floor(log2) - 2
    e = np.maximum(e, -127)
    v = np.abs(np.ldexp(b, -e[..., None]))
    # nearest code, the even one on a tie: compare with the midpoints
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    code = np.zeros(v.shape, np.int64)
    for i, m in enumerate(mid):
        code += (v >= m) if i % 2 == 1 else (v > m)
    code += np.where(np.signbit(w32.reshape(b.shape)), 8, 0)
    code = np.where(bad[..., None], 0, code)
    byte = np.where(bad, 255, e + 127)
    return code.reshape(n, k).astype(np.uint8), byte.astype(np.uint8)


def pack(code: np.ndarray) -> np.ndarray:
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def values(packed: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values [..., K]; a block of scale byte 255 is NaN."""
    c = np.empty((*packed.shape[:-1], packed.shape[-1] * 2), np.int64)
    c[..., 0::2] = packed & 15
    c[..., 1::2] = packed >> 4
    v = np.where(c >= 8, -1.0, 1.0) * E2M1[c & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def matmul(xq, xs, packed, scales):
    """(y, sum of |x w|), both float64 [M, N]."""
    x, w = values(xq, xs), values(packed, scales)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def grouped(x: np.ndarray, w: np.ndarray, offsets, y: np.ndarray):
    """Rows offsets[e] .. offsets[e+1]-1 of x times w[e]^T; the other rows are y's.
    Returns (y, sum of |x w|) in float64."""
    y = y.astype(np.float64).copy()
    mag = np.zeros_like(y)
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            y[a:b] = x[a:b] @ w[e].T
            mag[a:b] = np.abs(x[a:b]) @ np.abs(w[e]).T
    return y, mag
