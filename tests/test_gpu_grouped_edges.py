"""Edges of the products by expert: the shortest K of each unit of columns,
rows that hold no numbers, bounds out of order with bf16 x, and a first call
that is captured."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import tests.grouped_cases as GC
from tests.gpu_util import Canary
from tests.test_gpu_grouped_precision import product

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def w4():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import dequant_gemm_quantize_amd as m
    m.load()
    return m


@pytest.mark.parametrize("k,g", [(64, 64), (64, 32), (128, 128), (128, 64), (192, 192), (256, 128), (320, 32), (384, 128)])
@pytest.mark.parametrize("split", sorted(GC.SPLITS))
def test_short_rows_exact(w4, split, k, g):
    off, t = GC.offsets_of(split)
    x, code, s, z = GC.sparse_scales_f16(np.random.default_rng(k + g + t), t, len(off) - 1, 131, k, g)
    for out in ("bf16", "f32"):
        y = product(w4, x, code, s, z, g, off, out)
        want = torch.from_numpy(GC.exact(x, GC.weights(code, s, z, g), off, t, 131, -7.0)).to(y.dtype)
        assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("xd", ["bf16", "f32"])
@pytest.mark.parametrize("g", [32, 64, 128])
@pytest.mark.parametrize("split", sorted(GC.SPLITS))
def test_bad_rows_stay_alone(w4, split, g, xd):
    """Rows of x that no expert has, and one row of an expert, hold NaN and infinities: the other rows are exact."""
    off, t = GC.offsets_of(split)
    e, n, k = len(off) - 1, 70, 384
    x, code, s, z = GC.sparse_scales_f16(np.random.default_rng(g + t), t, e, n, k, g)
    bad = np.ones(t, bool)
    bad[off[0]:off[-1]] = False
    mine = int(off[-1]) - 1
    x[bad] = np.nan
    x[mine, ::3], x[mine, 1::3], x[mine, 2::3] = np.inf, -np.inf, np.nan
    y = product(w4, x, code, s, z, g, off, "f32", xd=xd).cpu()
    clean = x.copy()
    clean[mine], clean[bad] = 0, 0
    want = torch.from_numpy(GC.exact(clean, GC.weights(code, s, z, g), off, t, n, -7.0)).float()
    others = torch.ones(t, dtype=torch.bool)
    others[mine] = False
    assert torch.equal(y[others], want[others]) and torch.isnan(y[mine]).all()


@pytest.mark.parametrize("n", [130, 1000])
@pytest.mark.parametrize("cuts", [[0, 500, 100, 300], [-5, 20, 40, 1 << 30], [300, 200, 100, 0], [7, 7, 7, 7],
                                  [0, 300, 0, 300], [-(1 << 31), (1 << 31) - 1, -(1 << 31), (1 << 31) - 1]])
@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
def test_bounds_out_of_order_with_many_rows(w4, fmt, cuts, n):
    """As test_offsets_out_of_order_stay_in_bounds, in the many-row kernels: whatever is written lies inside y."""
    t, e, k = 300, 3, 256
    layer = w4.QuantizedExperts.from_weight(torch.randn((e, n, k), device="cuda") * 0.05, fmt=fmt)
    c = Canary((t, n), torch.bfloat16)
    c.tensor.fill_(-7.0)
    layer(torch.randn((t, k), device="cuda").to(torch.bfloat16), torch.tensor(cuts, dtype=torch.int32).cuda(), out=c.tensor)
    c.check()
    assert torch.isfinite(c.tensor).all()


CAPTURED = """
import torch
import dequant_gemm_quantize_amd as w4
t, e, n, k, fmt = 400, 2, 300, 256, {fmt!r}
x = torch.randn((t, k), device="cuda").to(torch.bfloat16)
layer = w4.QuantizedExperts.from_weight(torch.randn((e, n, k), device="cuda") * 0.05, fmt=fmt)
off = torch.tensor([0, 150, 400], dtype=torch.int32, device="cuda")
y = torch.zeros((t, n), dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    layer(x, off, out=y)
for _ in range(3):
    y.zero_()
    graph.replay()
    want = layer(x, off)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and y.float().abs().max() > 0
print("replayed")
"""


@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
def test_first_call_captured(fmt):
    """In a fresh process the first call of a many-row product is captured: its one-time setting is no stream operation."""
    r = subprocess.run([sys.executable, "-c", CAPTURED.format(fmt=fmt)], cwd=ROOT, capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "replayed" in r.stdout, r.stderr[-2000:]
