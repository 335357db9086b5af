"""Inputs and 64-bit definitions of the products with adapters, for the GPU tests.

Nothing here uses the library.  `whole` inputs are small whole numbers (and
powers of two for scales), so that every sum is a whole number of the smallest
unit below 2^24 of them: float32 results have no rounding at all, whatever the
order of the sums, and are compared bit for bit.
"""
from __future__ import annotations

import torch

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step, relative


def weight(n, k, g, sz, gen, whole):
    q = torch.randint(0, 16, (n, k), generator=gen, device=DEV, dtype=torch.uint8)
    packed = q[:, 0::2] | (q[:, 1::2] << 4)
    zeros = torch.randint(0, 16, (n, k // g), generator=gen, device=DEV).to(DT[sz])
    if whole:
        scales = (2.0 ** torch.randint(0, 2, (n, k // g), generator=gen, device=DEV)).to(DT[sz])
    else:
        scales = (torch.rand((n, k // g), generator=gen, device=DEV) * 0.01 + 0.001).to(DT[sz])
    dense = (q.double() - zeros.double().repeat_interleave(g, 1)) * scales.double().repeat_interleave(g, 1)
    return packed.contiguous(), scales, zeros, dense


def values(shape, dtype, gen, whole, most=1):
    if whole:
        return torch.randint(-most, most + 1, shape, generator=gen, device=DEV).to(dtype)
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def case(m, n, k, g, r, bounds, which, l, x="bf16", ab="bf16", sz="f16", whole=True, seed=0):
    """x [M, K], dy [M, N], a weight, L adapters and the segments (bounds, which: lists)."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    packed, scales, zeros, dense = weight(n, k, g, sz, gen, whole)
    c = {"m": m, "n": n, "k": k, "g": g, "r": r, "l": l, "weight": (packed, scales, zeros, g), "dense": dense,
         "x": values((m, k), DT[x], gen, whole), "dy": values((m, n), DT[x], gen, whole),
         "a": values((l, r, k), DT[ab], gen, whole), "b": values((l, n, r), DT[ab], gen, whole),
         "scaling": (2.0 ** torch.randint(-1, 2, (l,), generator=gen, device=DEV)).float() if whole
         else torch.rand((l,), generator=gen, device=DEV) + 0.5,
         "offsets": torch.tensor(bounds, dtype=torch.int32, device=DEV),
         "which": torch.tensor(which, dtype=torch.int32, device=DEV), "bounds": bounds, "ids": which}
    if not whole:
        c["a"], c["b"] = c["a"] * k ** -0.5, c["b"] * 0.02
        c["a"], c["b"] = c["a"].to(DT[ab]), c["b"].to(DT[ab])
    c["adapter"] = (c["a"], c["b"], c["scaling"], c["offsets"], c["which"])
    return c


def owned(c):
    """(rows, adapter) of the segments that have one."""
    return [(slice(lo, hi), i) for lo, hi, i in zip(c["bounds"], c["bounds"][1:], c["ids"]) if 0 <= i < c["l"] and hi > lo]


def forward64(c):
    x = c["x"].double()
    y, u = x @ c["dense"].t(), torch.zeros((c["m"], c["r"]), dtype=torch.float64, device=DEV)
    for rows, i in owned(c):
        u[rows] = c["scaling"][i].double() * (x[rows] @ c["a"][i].double().t())
        y[rows] += u[rows] @ c["b"][i].double().t()
    return y, u


def back64(c):
    dy = c["dy"].double()
    dx, v = dy @ c["dense"], torch.zeros((c["m"], c["r"]), dtype=torch.float64, device=DEV)
    for rows, i in owned(c):
        v[rows] = c["scaling"][i].double() * (dy[rows] @ c["b"][i].double())
        dx[rows] += v[rows] @ c["a"][i].double()
    return dx, v


def grads64(c, xhat, u, v):
    da = torch.zeros((c["l"], c["r"], c["k"]), dtype=torch.float64, device=DEV)
    db = torch.zeros((c["l"], c["n"], c["r"]), dtype=torch.float64, device=DEV)
    for rows, i in owned(c):
        da[i] += v[rows].double().t().contiguous() @ xhat[rows]
        db[i] += c["dy"][rows].double().t().contiguous() @ u[rows].double()
    return da, db


def sum_tol(n):
    """Relative 2-norm error of a float32 sum of n random terms: each addition rounds
    the running sum by half a step at most, 2^-24 of it; sums of i terms are
    sqrt(i) of one, so independent roundings leave 2^-24 sqrt(n / 2) of the sum; twice
    sqrt(n) is nearly three times that, and 4 more steps cover products, scales and joins."""
    return (2 * n ** 0.5 + 4) * 2.0 ** -24


def rel(got, want):
    return float((got.double() - want).norm() / want.norm().clamp(min=1e-300))
