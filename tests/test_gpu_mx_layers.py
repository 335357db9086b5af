"""The MXFP4 layers in the place of dense ones: results come in x's own type,
so a model whose other layers stayed dense still runs, in every float type."""
import numpy as np
import pytest
import torch

import oracle.mxfp4_oracle as MX
from tests.gpu_util import to_host

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def w4():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import dequant_gemm_quantize_amd as m
    m.load()
    return m


@pytest.mark.parametrize("dt", DTYPES)
def test_model_with_dense_layers_left(w4, dt):
    """A layer with a bias stays dense and takes what the replaced one in front of it gives."""
    torch.manual_seed(1)
    model = torch.nn.Sequential(torch.nn.Linear(64, 96, bias=False), torch.nn.ReLU(), torch.nn.Linear(96, 10)).cuda().to(dt)
    w4.replace_linears(model, mode="mxfp4")
    assert type(model[0]).__name__ == "MXFP4Linear" and type(model[2]) is torch.nn.Linear
    x = torch.randn(5, 64, device="cuda").to(dt)
    with torch.no_grad():
        y = model(x)
        h = model[0](x)
    assert h.dtype == dt and y.dtype == dt
    ref, mag = product(w4, x, model[0])
    # the products are exact in float32 and 64 additions are off by 2^-23 of their sum at most; then one rounding to dt
    tol = 64 * 2.0 ** -23 * mag
    tol = tol if dt == torch.float32 else tol * 2 + torch.finfo(dt).eps * np.abs(ref) + 2.0 ** -24
    assert (np.abs(h.double().cpu().numpy() - ref) <= tol).all()


def product(w4, x, layer):
    c, s = MX.quantize(x.float().cpu().numpy())
    return MX.matmul(MX.pack(c), s, to_host(layer.packed), to_host(layer.scales))


@pytest.mark.parametrize("fmt", ["mxfp4", "int4"])
@pytest.mark.parametrize("dt", DTYPES)
def test_experts_give_the_type_they_take(w4, fmt, dt):
    e, n, k = 3, 40, 128
    layer = w4.QuantizedExperts.from_weight(torch.randn((e, n, k), device="cuda") * 0.05, fmt=fmt)
    off = torch.tensor([0, 4, 4, 9], dtype=torch.int32, device="cuda")
    x = torch.randn((9, k), device="cuda").to(dt)
    y = layer(x, off)
    assert y.dtype == dt and y.shape == (9, n)
    # in float32 the same call gives what y is the rounding of
    full = torch.empty((9, n), dtype=torch.float32, device="cuda")
    layer(x, off, out=full)
    assert torch.equal(y, full.to(dt))


@pytest.mark.parametrize("out", DTYPES)
def test_out_dtype_is_kept(w4, out):
    layer = w4.MXFP4Linear.from_weight(torch.randn((40, 64), device="cuda") * 0.05, out_dtype=out)
    for dt in DTYPES:
        assert layer(torch.randn((3, 64), device="cuda").to(dt)).dtype == out
