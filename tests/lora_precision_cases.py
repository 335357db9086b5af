"""Cases of the products with adapters and of the transposed product whose results show whether a weight was rounded on
the way, the allowances of their results, and models of the rounding.  Nothing here uses the library; every function
runs on the CPU and on a GPU alike."""
from __future__ import annotations

import torch

# rows, out, in, group.  Forward: what many rows take (above 64 rows and 2^31 products), by groups of a multiple
# of 128, 64 and 32 columns, K that ends inside a step of 64 columns, tiles of 128 and 64 rows, sums in one part and in
# several; then few rows.
FORWARD = [(300, 2056, 4096, 128), (1100, 2050, 1024, 128), (130, 4104, 4224, 384), (200, 2100, 5184, 64), (1100, 700, 2880, 32),
           (700, 1032, 3040, 32), (140, 5000, 3168, 96), (60, 300, 1024, 128), (3, 130, 576, 192)]
# Back: tiles (above 32 rows, N a multiple of 8) of 256 and 128 rows, groups of a multiple of 128 columns and others,
# split sums; then few rows, in one block of 16 and two, and N that is no multiple of 8.
BACK = [(300, 2056, 4096, 128), (1100, 1032, 1024, 256), (100, 4104, 2112, 64), (270, 520, 960, 32), (40, 808, 1056, 96),
        (12, 1000, 2048, 128), (32, 640, 768, 32), (90, 333, 512, 64)]


def bf16(a):
    return a.to(torch.bfloat16).to(a.dtype)


def in_two(w):
    """The weight as the sum of two bf16 values."""
    hi = bf16(w)
    return hi + bf16(w - hi)


def sparse(rows, columns, count, most, gen):
    """[rows, columns] of zeros but for `count` columns a row, whole numbers 1 .. most of either sign."""
    at = torch.rand((rows, columns), generator=gen).topk(count, 1).indices
    v = torch.randint(1, most + 1, (rows, count), generator=gen) * (2 * torch.randint(0, 2, (rows, count), generator=gen) - 1)
    return torch.zeros((rows, columns)).scatter_(1, at, v.float())


def case(m, n, k, g, sz, dev, seed):
    """A weight whose values need more bits than bf16 has, x and dy of three columns a row, and two adapters of whole
    numbers for the second half of the rows (rank 8).

    sz f16: scales of 11 bits, 1/8 .. 1/4 in steps of 2^-13, so that products and sums are multiples of 2^-13: up
    to 9 . 16 / 4 of the weight, with 31 in place of 15 below 2^7, and 8 . 9 . 2 from the adapters: below 2^9 in all, exact in float32 in any order.
    sz f32: scales of 24 bits, the lowest of them set, and weights of 12 to 15 scales."""
    gen = torch.Generator().manual_seed(seed)
    shape = (n, k // g)
    if sz == "f16":
        s = (torch.randint(1024, 2048, shape, generator=gen) / 2.0 ** 13).to(torch.float16)
        z = torch.randint(0, 16, shape, generator=gen)
        q = torch.randint(0, 16, (n, k), generator=gen)
    else:
        s = ((torch.randint(1 << 22, 1 << 23, shape, generator=gen) * 2 + 1).double() / 2.0 ** 26).float()
        high = torch.randint(0, 2, shape, generator=gen)
        z = torch.where(high == 1, 15, torch.randint(0, 2, shape, generator=gen))
        q = torch.where(high.repeat_interleave(g, 1) == 1, torch.randint(0, 4, (n, k), generator=gen),
                        torch.randint(13, 16, (n, k), generator=gen))
    q = q.to(torch.uint8)
    c = {"m": m, "n": n, "k": k, "g": g, "sz": sz}
    c["packed"], c["scales"], c["zeros"] = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), s, z.to(s.dtype)
    c["dense"] = (q.double() - z.double().repeat_interleave(g, 1)) * s.double().repeat_interleave(g, 1)
    c["x"], c["dy"] = sparse(m, k, 3, 3, gen), sparse(m, n, 3, 3, gen)
    c["a"], c["b"] = torch.randint(-1, 2, (2, 8, k), generator=gen).float(), torch.randint(-1, 2, (2, n, 8), generator=gen).float()
    c["scaling"] = torch.tensor([2.0, 0.5])
    c["bounds"], c["ids"] = [m // 2, 3 * m // 4, m], [1, 0]
    c = {name: t.to(dev) if isinstance(t, torch.Tensor) else t for name, t in c.items()}
    for name, t in (("offsets", c["bounds"]), ("which", c["ids"])):
        c[name] = torch.tensor(t, dtype=torch.int32, device=dev)
    return c


def forward(c, dense):
    y = c["x"].double() @ dense.t()
    for lo, hi, i in zip(c["bounds"], c["bounds"][1:], c["ids"]):
        u = c["scaling"][i].double() * (c["x"][lo:hi].double() @ c["a"][i].double().t())
        y[lo:hi] += u @ c["b"][i].double().t()
    return y


def back(c, dense):
    dx = c["dy"].double() @ dense
    for lo, hi, i in zip(c["bounds"], c["bounds"][1:], c["ids"]):
        v = c["scaling"][i].double() * (c["dy"][lo:hi].double() @ c["b"][i].double())
        dx[lo:hi] += v @ c["a"][i].double()
    return dx


def magnitude(c, transposed):
    """Sums of |x| s: what one unit of the codes counts for in each result; the adapters' sums, up to 8 . 9 . 2, added."""
    s = c["scales"].double().repeat_interleave(c["g"], 1)
    mag = c["dy"].double().abs() @ s if transposed else c["x"].double().abs() @ s.t()
    mag[c["bounds"][0]:] += 144
    return mag


def allowance(c, transposed, out, want):
    """How far the result may be off.  float32, whatever the form: every product (up to 31 |x| s) and every sum of the few
    terms is off by half a step: products of codes and zero-points, 31 each, the sums of the parts of one and the
    joins of both, six more of 31 at most.  Back, a bf16 result of float32 scales has weights of 16 bits: up
    to 15 scales, off by 2^-16 of them.  A bf16 result is rounded once more, by half a step of its binade (eight bits)."""
    mag = magnitude(c, transposed)
    allowed = 2.0 ** -24 * 8 * 31 * mag
    if out == torch.bfloat16:
        if transposed and c["sz"] == "f32":
            allowed = allowed + 2.0 ** -16 * 15 * mag
        allowed = allowed + torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -100))) - 8) * (1 + 2.0 ** -7)
    return allowed
