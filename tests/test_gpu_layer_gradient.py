"""The gradient through a frozen QuantizedLinear: against the formula and against differences, in a model beside a
residual path, with odd widths and other types of the result."""
import pytest
import torch

import dequant_gemm_quantize_amd as w4
from tests import lora_cases as C

pytestmark = pytest.mark.gpu


def layer(n, k, g=64, **kw):
    gen = torch.Generator(device="cuda").manual_seed(n + k)
    return w4.QuantizedLinear.from_weight(torch.randn((n, k), generator=gen, device="cuda") * 0.05, group_size=g, **kw)


@pytest.mark.parametrize("dtype,out", [(torch.float32, None), (torch.bfloat16, None), (torch.bfloat16, torch.float32),
                                       (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("lead,n,k", [((1,), 96, 256), ((3, 4), 101, 128), ((150,), 1024, 192), ((2, 40), 200, 448)])
def test_against_the_formula(lead, n, k, dtype, out):
    one = layer(n, k, out_dtype=out)
    x = torch.randn(*lead, k, device="cuda").to(dtype).requires_grad_()
    y = one(x)
    with torch.no_grad():
        plain = one(x)
    assert plain.grad_fn is None and torch.equal(y, plain) and y.dtype == (out or dtype)
    dy = torch.randn_like(y)
    dx, = torch.autograd.grad(y, x, dy)
    want = dy.double().reshape(-1, n) @ one.dequantize(torch.float32).double()
    # one rounding of the result, half a step of each element at most, beside float32 sums
    assert dx.dtype == dtype and dx.shape == x.shape
    assert C.rel(dx.reshape(-1, k), want) <= C.HALF[dtype] + C.sum_tol(n)


def test_against_differences():
    """The loss is linear in x: a difference quotient is its derivative but for the roundings of the two losses, 2^-24
    sqrt(n) of sums of n terms each (sum_tol), relative to the loss's size over the step's."""
    one = layer(96, 256)
    x = torch.randint(-9, 10, (20, 256), device="cuda").float().requires_grad_()
    dy = torch.randn(20, 96, device="cuda")
    dx, = torch.autograd.grad(one(x), x, dy)
    step = torch.randint(-3, 4, x.shape, device="cuda").float()
    with torch.no_grad():
        losses = [(one(x + sign * step).double() * dy.double()).sum() for sign in (1, -1)]
        size = (one(x).double() * dy.double()).abs().sum() + sum(abs(v) for v in losses)
    slope, want = (losses[0] - losses[1]) / 2, (dx.double() * step.double()).sum()
    assert float((slope - want).abs()) <= 4 * C.sum_tol(256) * float(size) + 1e-6 * float(want.abs())


class Block(torch.nn.Module):
    def __init__(self, width):
        super().__init__()
        self.into = torch.nn.Linear(width, width)
        self.up, self.down = torch.nn.Linear(width, 3 * width, bias=False), torch.nn.Linear(3 * width, width, bias=False)

    def forward(self, x):
        x = self.into(x)
        return x + self.down(torch.relu(self.up(x)))


def test_a_model_with_a_residual_path():
    """Frozen projections beside a residual: the gradient that reaches the layer before them is that of the dense model
    with the same weights."""
    torch.manual_seed(1)
    model = Block(128).cuda()
    w4.replace_linears(model, group_size=32, skip=lambda name, m: name == "into")
    dense = Block(128).cuda()
    with torch.no_grad():
        dense.into.weight.copy_(model.into.weight), dense.into.bias.copy_(model.into.bias)
        for name in ("up", "down"):
            getattr(dense, name).weight.copy_(getattr(model, name).dequantize(torch.float32))
    x = torch.randn(10, 128, device="cuda")
    dy = torch.randn(10, 128, device="cuda")
    got = torch.autograd.grad(model(x), model.into.weight, dy)[0]
    want = torch.autograd.grad(dense.double()(x.double()), dense.into.weight, dy.double())[0]
    assert C.rel(got, want) <= 4 * (C.sum_tol(128) + C.sum_tol(384)) + 1e-5  # a relu's side may turn within float32


def test_adapters_behind_a_frozen_layer():
    """Adapters on one projection only: their gradients pass the frozen one behind them."""
    torch.manual_seed(2)
    lora = w4.LoRALinear(layer(192, 128), rank=8)
    frozen = layer(64, 192)
    with torch.no_grad():
        lora.b.copy_(torch.randn_like(lora.b) * 0.1)
    x = torch.randn(9, 128, device="cuda")
    da, db = torch.autograd.grad(frozen(lora(x)).sum(), (lora.a, lora.b))
    assert da.abs().max() > 0 and db.abs().max() > 0


def test_views_and_no_second_derivative():
    one = layer(101, 128)
    x = torch.randn(8, 128, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    dy = torch.randn(8, 101, device="cuda").bfloat16()
    want, = torch.autograd.grad(one(x), x, dy)
    got, = torch.autograd.grad(torch.cat([one(x[:3]), one(x[3:])]), x, dy)
    assert torch.equal(got, want)
    dx, = torch.autograd.grad(one(x).float().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()
    empty = torch.randn(0, 128, device="cuda", requires_grad=True)
    assert torch.autograd.grad(one(empty).sum(), empty)[0].shape == (0, 128)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_layers_of_many_rows(dtype):
    """Adapters of several requests, then a frozen layer of an odd width, at sizes that take the many-row kernels: every
    gradient against the formula in 64 bits at the values that the layers passed on."""
    torch.manual_seed(3)
    m, k, h, n = 900, 1280, 2048, 1033
    lora, frozen = w4.LoRALinear(layer(h, k, 128), rank=24, adapters=3, dtype=torch.float32), layer(n, h, 128)
    with torch.no_grad():
        lora.b.copy_(torch.randn_like(lora.b) * 0.1)
    offsets = torch.tensor([0, 100, 777, m], dtype=torch.int32, device="cuda")
    which = torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    x = torch.randint(-126, 127, (m, k), device="cuda").to(dtype)  # whole numbers, 127 the largest of each block: kept exactly in 8 bits
    x[:, ::128] = 127
    x.requires_grad_()
    z = lora(x, offsets, which)
    y = frozen(z)
    dy = (torch.randn(m, n, device="cuda") * 1e-2).to(dtype)
    dx, dz, da, db = torch.autograd.grad(y, (x, z, lora.a, lora.b), dy)
    w1 = w4.QuantizedLinear(k, h, 128, device="cuda")
    w1.packed, w1.scales, w1.zeros = lora.packed, lora.scales, lora.zeros
    w1, w2 = w1.dequantize(torch.float32).double(), frozen.dequantize(torch.float32).double()
    assert C.rel(dz, dy.double() @ w2) <= C.HALF[dtype] + C.sum_tol(n)
    d, a, b = dz.double(), lora.a.detach().double(), lora.b.detach().double()
    want_x, want_a, want_b = d @ w1, torch.zeros_like(a), torch.zeros_like(b)
    for rows, l in ((slice(0, 100), 2), (slice(777, m), 0)):
        u, v = x[rows].detach().double() @ a[l].t(), d[rows] @ b[l]
        want_x[rows] += v @ a[l]
        want_a[l], want_b[l] = v.t().contiguous() @ x[rows].detach().double(), d[rows].t().contiguous() @ u
    assert C.rel(dx, want_x) <= C.HALF[dtype] + 4 * C.sum_tol(h)
    assert C.rel(da, want_a) <= 4 * C.sum_tol(h) and C.rel(db, want_b) <= 4 * C.sum_tol(k)
    assert not da[1].any() and not db[1].any()
