"""MXFP4 products with block scales at the ends of their range, in both kernels
of each form: NaN scales reach their own row or column and nothing else, also
where a row's last step reads into the next row, and scales whose products
leave float32's normal range.

Finite results are exact (tests/test_gpu_mxfp4.py): scale bytes 126..128.
"""
import numpy as np
import pytest
import torch

import oracle.mxfp4_oracle as MX
from tests.gpu_util import Canary, to_dev
from tests.test_gpu_mxfp4 import dev, exact_operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import dequant_gemm_quantize_amd as m
    m.load()
    return m


def mark(rng, scales, rows):
    """Byte 255 in one block of each of these rows: the first, the last, then any."""
    for i, r in enumerate(rows):
        scales[r, 0 if i == 0 else scales.shape[1] - 1 if i == 1 else rng.integers(0, scales.shape[1])] = 255


def same(y, want):
    """Equal, NaN included."""
    want = torch.from_numpy(want).to(y.dtype)
    got = y.cpu()
    return torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(4, 70, 96), (20, 300, 544), (64, 5000, 128), (300, 513, 384), (300, 513, 128),
                                   (300, 260, 160), (700, 5001, 640), (1500, 4100, 384)])
def test_nan_scales_stay_in_their_rows(w4, m, n, k, out):
    rng = np.random.default_rng(m + n + k)
    x, w = exact_operand(rng, m, k), exact_operand(rng, n, k)
    xr, wr = [1, m // 2, m - 1], [0, 5, n // 3, n - 2]
    mark(rng, x[1], xr), mark(rng, w[1], wr)
    c = Canary((m, n), torch.float32 if out == "f32" else torch.bfloat16)
    w4.mxfp4_matmul(*dev(x), *dev(w), out=c.tensor)
    c.check()
    want = MX.matmul(*x, *w)[0]
    nan = np.isnan(want)
    assert nan[xr].all() and nan[:, wr].all() and not np.delete(np.delete(nan, xr, 0), wr, 1).any()
    assert same(c.tensor, want)


@pytest.mark.parametrize("n,k", [(130, 128), (70, 96), (300, 384), (130, 640)])
@pytest.mark.parametrize("sizes", [[0, 2, 0, 1, 1, 0], [70, 0, 129, 33, 1, 256], [600, 500]])
def test_nan_scales_by_expert(w4, sizes, n, k):
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    t, e = int(off[-1]), len(sizes)
    rng = np.random.default_rng(n + k + t)
    x, w = exact_operand(rng, t, k), exact_operand(rng, e * n, k)
    mark(rng, x[1], [0, t // 2]), mark(rng, w[1], [n - 1, n, 2 * n + 3] if e > 2 else [n - 1, n])
    wq, ws = w[0].reshape(e, n, -1), w[1].reshape(e, n, -1)
    c = Canary((t, n), torch.float32)
    w4.mxfp4_grouped_matmul(*dev(x), torch.from_numpy(off).cuda(), to_dev(wq, "u8"), to_dev(ws, "u8"), out=c.tensor)
    c.check()
    want, _ = MX.grouped(MX.values(*x), MX.values(wq, ws), off, np.zeros((t, n)))
    assert 0 < np.isnan(want).sum() < want.size
    assert same(c.tensor, want)


@pytest.mark.parametrize("total", [254 - 130, 254 - 140, 254 - 147])
@pytest.mark.parametrize("m,k", [(3, 544), (300, 384), (300, 160)])
def test_subnormal_results_exact(w4, m, k, total):
    """Scale bytes that add up to `total` in every block: products are multiples of 2^-2 2^(total - 254) >= 2^-149, sums
    below 2^24 of them."""
    rng = np.random.default_rng(m + k + total)
    n = 140
    x, w = exact_operand(rng, m, k), exact_operand(rng, n, k)
    x[1][:], w[1][:] = np.arange(k // 32) % 3 + 40, total - 40 - np.arange(k // 32) % 3
    want = MX.matmul(*x, *w)[0]
    y = w4.mxfp4_matmul(*dev(x), *dev(w), out_dtype=torch.float32)
    assert np.abs(want).max() < 2.0 ** (total - 254 - 2 + 24) and want.any()
    assert torch.equal(y.cpu(), torch.from_numpy(want).float())


@pytest.mark.parametrize("total", [0, 40, 80])
@pytest.mark.parametrize("m,k", [(3, 544), (300, 384), (300, 160)])
def test_tiny_products_vanish(w4, m, k, total):
    """Sums of K products of 36 2^(80 - 254) at most, far below 2^-150, leave zero and change nothing beside others."""
    rng = np.random.default_rng(m + k + total)
    n = 140
    x, w = exact_operand(rng, m, k), exact_operand(rng, n, k)
    x[1][:], w[1][:] = total // 2, total - total // 2
    y = w4.mxfp4_matmul(*dev(x), *dev(w), out_dtype=torch.float32)
    assert not y.any()
    x[1][:, -1], w[1][:, -1] = 127, 127  # one block of the row counts
    y = w4.mxfp4_matmul(*dev(x), *dev(w), out_dtype=torch.float32)
    last = [MX.values(o[0][:, -16:], o[1][:, -1:]) for o in (x, w)]
    assert torch.equal(y.cpu(), torch.from_numpy(last[0] @ last[1].T).float())
