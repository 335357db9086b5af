"""Cases of the INT4 product by expert whose result shows whether a weight, a
scale or a part of x was rounded on the way, and NumPy models of the product.

Everything here is NumPy on the CPU; nothing is shared with the HIP path.
"""
import numpy as np

import oracle.mxfp4_oracle as MX

# (rows of each expert, rows before the first, rows behind the last)
SPLITS = {
    "few": ([0, 2, 0, 1, 1, 0], 0, 0),
    "some": ([3, 0, 17, 16, 40], 4, 7),
    "many": ([70, 0, 129, 33, 1, 256], 1, 30),
    "most": ([600, 500], 0, 3),
}
# N, K, group: units of 128, 64 and 32 columns, whole and partial pairs of them, groups of several units
SHAPES = [(130, 512, 128), (65, 640, 128), (70, 768, 384), (129, 448, 64), (70, 320, 64), (33, 576, 192), (200, 704, 32),
          (64, 960, 96)]


def offsets_of(split):
    sizes, before, behind = SPLITS[split]
    off = np.concatenate([[0], np.cumsum(sizes)]) + before
    return off.astype(np.int32), int(off[-1]) + behind


def bf16(a):
    """float32 values of a rounded to bfloat16, nearest even (finite values)."""
    u = np.ascontiguousarray(a, np.float32).view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def sparse(rng, t, k, count, values):
    """[t, k] of zeros but for `count` columns a row, which hold one of `values` or its negative."""
    x = np.zeros((t, k), np.float32)
    for r in range(t):
        x[r, rng.choice(k, count, replace=False)] = rng.choice(values, count) * rng.choice([-1, 1], count)
    return x


def sparse_scales_f16(rng, t, e, n, k, g):
    """x of three columns, scales of 11 significant bits.  Every product and sum is a multiple of 2^-13 below 2^7, so
    exact in float32 in any order: a result equals the rounding of the exact one, unless a weight was rounded before."""
    x = sparse(rng, t, k, 3, [1.0, 2.0, 3.0])
    code = rng.integers(0, 16, (e, n, k)).astype(np.uint8)
    s = (rng.integers(1024, 2048, (e, n, k // g)) / 2.0 ** 13).astype(np.float32)
    z = rng.integers(0, 16, (e, n, k // g)).astype(np.float32)
    return x, code, s, z


def sparse_scales_f32(rng, t, e, n, k, g):
    """x of one column, scales of 24 significant bits, and weights of 12 to 15 scales."""
    x = sparse(rng, t, k, 1, [1.0, 2.0])
    s = ((rng.integers(1 << 22, 1 << 23, (e, n, k // g)) * 2 + 1) / 2.0 ** 26).astype(np.float32)
    high = rng.integers(0, 2, (e, n, k // g))
    z = np.where(high, 15, rng.integers(0, 2, (e, n, k // g))).astype(np.float32)
    code = np.where(np.repeat(high, g, -1), rng.integers(0, 4, (e, n, k)), rng.integers(13, 16, (e, n, k)))
    return x, code.astype(np.uint8), s, z


def weights(code, s, z, g):
    """(q - zp) s in float64."""
    return (code.astype(np.float64) - np.repeat(z, g, -1)) * np.repeat(s, g, -1).astype(np.float64)


def exact(x, w, off, t, n, fill=0.0):
    return MX.grouped(x.astype(np.float64), w, off, np.full((t, n), fill))[0]


def allowance_f32(x, s, g, off):
    """How far a float32 result of sparse_scales_f32 may be off.  With one column x of scale s: the products s x (16 + q)
    and s x (16 + zp), or s x q and s zp, are off by half a step each (2^-24 of up to 31 |x| s and 31 |x| s), and the
    scaled sum and the zero-point's three parts are added with half a step of at most 30 |x| s each time."""
    mag = MX.grouped(np.abs(x).astype(np.float64), np.repeat(s, g, -1).astype(np.float64), off,
                     np.zeros((x.shape[0], s.shape[1])))[0]
    return 2.0 ** -24 * (31 + 31 + 3 * 30) * mag


def wide_x(rng, t, e, n, k, g):
    """float32 x of two columns, whole numbers of 17 bits whose bits 16, 8 and 0 are set: each bf16 part, of 8 bits from
    its highest on, leaves something for the next.  The scale is 1/2, so every product and sum, with 16 + code too, is a
    multiple of 1/2 below 2^22 (2 2^17 31 / 2): exact in float32 in any order."""
    values = np.array([1 << 16 | a << 9 | 1 << 8 | b << 1 | 1 for a in range(0, 128, 9) for b in range(0, 128, 11)])
    x = sparse(rng, t, k, 2, values.astype(np.float32))
    code = rng.integers(0, 16, (e, n, k)).astype(np.uint8)
    s = np.full((e, n, k // g), 0.5, np.float32)
    z = rng.integers(0, 16, (e, n, k // g)).astype(np.float32)
    return x, code, s, z


def parts(x):
    """float32 x as hi + mid + lo, each the upper half of what is left."""
    out = []
    left = np.ascontiguousarray(x, np.float32)
    for _ in range(3):
        p = (left.view(np.uint32) & 0xFFFF0000).astype(np.uint32).view(np.float32)
        out.append(p)
        left = left - p
    assert not left.any()
    return out


def real_float_x(rng, t, e, n, k):
    x = rng.normal(0, 1, (t, k)).astype(np.float32)
    return x, rng.normal(0, 0.02, (e * n, k)).astype(np.float32)


def allowance_real(x, s, g, off):
    """How far a float32 result of normal data may be off, growing with the root of the additions.  A matrix instruction
    adds 32 products at a time or more and a group's sum is added once, for codes and zero-points each: K / 32 + 2 K / g
    roundings, independent and of half a step of a partial sum each.  Partial sums are of terms up to 31 |x| s of any
    sign, root of the sum of their squares; 8 covers the largest of many outputs and the order inside an instruction."""
    k = x.shape[1]
    sq = MX.grouped(x.astype(np.float64) ** 2, (31 * np.repeat(s, g, -1).astype(np.float64)) ** 2, off,
                    np.zeros((x.shape[0], s.shape[1])))[0]
    return 8 * 2.0 ** -24 * np.sqrt(k / 32 + 2 * k / g) * np.sqrt(sq)
