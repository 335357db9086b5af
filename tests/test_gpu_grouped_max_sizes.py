"""The MXFP4 products and the products by expert at the largest sizes they take:
K = 2^23 columns, the last K of the INT4 many-row kernel and the first behind
it, T = 2^24 rows, 65536 experts.  Sampled rows against the oracle, bit for bit:

* MXFP4 with scale bytes 126..128: multiples of 2^-4; a sum of 2^23 such products is
  of the order of 2^16 (12 times the root of 2^23), far below the 2^20 up to which
  float32 holds them.
* INT4 with x in -1, 0, 1 and scales 2^-3..1: multiples of 2^-3, with 16 + code sums of
  the order of 2^17, far below 2^21.
"""
import numpy as np
import pytest
import torch

import oracle.mxfp4_oracle as MX

pytestmark = pytest.mark.gpu

MAX_K = 1 << 23


@pytest.fixture(scope="module")
def w4():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import dequant_gemm_quantize_amd as m
    m.load()
    return m


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def mx_operand(gen, rows, k):
    code = torch.randint(0, 256, (rows, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
    return code, torch.randint(126, 129, (rows, k // 32), dtype=torch.uint8, device="cuda", generator=gen)


def int4_weights(gen, e, n, k, g, sz=torch.float16):
    code = torch.randint(0, 256, (e, n, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scale = (0.125 * 2.0 ** torch.randint(0, 4, (e, n, k // g), device="cuda", generator=gen)).to(sz)
    return code, scale, torch.randint(0, 16, (e, n, k // g), device="cuda", generator=gen).to(sz)


def host(t):
    return t.cpu().numpy()


def int4_values(code, scale, zero, g):
    c = np.empty((*code.shape[:-1], code.shape[-1] * 2), np.float64)
    c[..., 0::2], c[..., 1::2] = code & 15, code >> 4
    return (c - np.repeat(zero.astype(np.float64), g, -1)) * np.repeat(scale.astype(np.float64), g, -1)


@pytest.mark.parametrize("m,k", [(3, MAX_K), (300, MAX_K), (300, MAX_K - 128), (20, MAX_K - 32)])
def test_mxfp4_longest_rows(w4, m, k):
    gen = generator(m)
    x, w = mx_operand(gen, m, k), mx_operand(gen, 3, k)
    y = w4.mxfp4_matmul(*x, *w, out_dtype=torch.float32)
    rows = [0, m - 1]
    want = MX.values(host(x[0][rows]), host(x[1][rows])) @ MX.values(*map(host, w)).T
    assert np.array_equal(host(y[rows]), want.astype(np.float32))


def test_quantize_longest_rows(w4):
    x = torch.randn((2, MAX_K), device="cuda", generator=generator(1)).to(torch.bfloat16)
    p, s = w4.quantize_mxfp4(x)
    code, byte = MX.quantize(host(x.float()))
    assert np.array_equal(host(s), byte) and np.array_equal(host(p), MX.pack(code))
    v = w4.dequant_mxfp4(p, s, out_dtype=torch.float32)
    assert np.array_equal(host(v), MX.values(host(p), host(s)).astype(np.float32))


@pytest.mark.parametrize("xd", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,k,g", [(5, MAX_K, 128), (70, 1 << 21, 128), (70, 1 << 21, 32), (70, 1 << 21, 1 << 21),
                                      (70, (1 << 21) + 64, 64), (3, MAX_K, MAX_K)])
def test_int4_longest_rows(w4, rows, k, g, xd):
    """2^21 columns are the many-row kernel's last, for bf16 x."""
    gen = generator(rows)
    e, n = 2, 3
    t = 2 * rows
    x = torch.randint(-1, 2, (t, k), device="cuda", generator=gen).to(xd)
    code, scale, zero = int4_weights(gen, e, n, k, g)
    off = torch.tensor([0, rows, t], dtype=torch.int32, device="cuda")
    y = w4.w4a16_grouped_matmul(x, off, code, scale, zero, g, out_dtype=torch.float32)
    for row, expert in ((0, 0), (rows, 1), (t - 1, 1)):
        w = int4_values(host(code[expert]), host(scale[expert]), host(zero[expert]), g)
        want = w @ host(x[row].double())
        assert np.array_equal(host(y[row]), want.astype(np.float32))


def cuts(t, e, seed):
    """Row bounds of e experts, some of them empty, and two rows that no expert has at either end."""
    rng = np.random.default_rng(seed)
    inner = np.sort(rng.integers(2, t - 1, e - 1)) if e > 1 else np.zeros(0, np.int64)
    return np.concatenate([[2], inner, [t - 2]]).astype(np.int32)


@pytest.mark.parametrize("fmt,k", [("mxfp4", 128), ("mxfp4", 96), ("int4", 64), ("int4", 32)])
@pytest.mark.parametrize("e", [1, 3, 65536])
def test_most_rows(w4, fmt, k, e):
    """2^24 rows; K decides between the many-row kernel and the few-row one."""
    t, n = 1 << 24, 5
    gen = generator(e + k)
    off = cuts(t, e, e)
    offd = torch.from_numpy(off).cuda()
    y = torch.full((t, n), -7.0, device="cuda")
    if fmt == "mxfp4":
        x = mx_operand(gen, t, k)
        code, scale = mx_operand(gen, e * n, k)
        code, scale = code.view(e, n, -1), scale.view(e, n, -1)
        w4.mxfp4_grouped_matmul(*x, offd, code, scale, out=y)
    else:
        x = torch.randint(-1, 2, (t, k), device="cuda", generator=gen, dtype=torch.int8).to(torch.bfloat16)
        code, scale, zero = int4_weights(gen, e, n, k, 32)
        w4.w4a16_grouped_matmul(x, offd, code, scale, zero, 32, out=y)
    rng = np.random.default_rng(e)
    rows = np.unique(np.concatenate([[0, 1, 2, 3, t - 3, t - 2, t - 1], rng.integers(0, t, 400), off[rng.integers(0, e, 50)]]))
    rows = rows[rows < t]
    owner = np.searchsorted(off, rows, side="right") - 1
    own = (owner >= 0) & (owner < e)
    idx = torch.from_numpy(rows).cuda()
    ex = torch.from_numpy(np.where(own, owner, 0)).cuda()
    if fmt == "mxfp4":
        xv, w = MX.values(host(x[0][idx]), host(x[1][idx])), MX.values(host(code[ex]), host(scale[ex]))
    else:
        xv, w = host(x[idx].double()), int4_values(host(code[ex]), host(scale[ex]), host(zero[ex]), 32)
    want = np.where(own[:, None], np.einsum("rk,rnk->rn", xv, w), -7.0)
    assert np.array_equal(host(y[idx]), want.astype(np.float32))
