"""The adapters' layer on tensors that are views into larger ones: gradients and activations that begin at any element."""
import pytest
import torch

import dequant_gemm_quantize_amd as w4

pytestmark = pytest.mark.gpu


def layer(n, k, dtype):
    torch.manual_seed(0)
    base = w4.QuantizedLinear.from_weight(torch.randn(n, k, device="cuda") * 0.05, group_size=32)
    lora = w4.LoRALinear(base, rank=8, dtype=dtype)
    with torch.no_grad():
        lora.b.copy_(torch.randn_like(lora.b) * 0.1)
    return lora


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [2050, 101])
def test_gradients_of_joined_results(n, dtype):
    """The backward of a concatenation hands on dense rows that begin at any element of the whole gradient."""
    lora = layer(n, 256, torch.float32)
    x = torch.randn(8, 256, device="cuda").to(dtype)
    parts = [x[:3].clone().requires_grad_(), x[3:].clone().requires_grad_()]
    dy = torch.randn(8, n, device="cuda").to(dtype)
    assert dy[3:].is_contiguous() and dy[3:].data_ptr() % 16 != 0
    z = torch.cat([lora(p) for p in parts])
    got = torch.autograd.grad(z, (*parts, lora.a, lora.b), dy)
    want = [torch.autograd.grad(lora(p), (p, lora.a, lora.b), d.clone()) for p, d in zip(parts, (dy[:3], dy[3:]))]
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[1][0])
    for g, a, b in zip(got[2:], want[0][1:], want[1][1:]):
        assert torch.equal(g, a + b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.float16])
def test_activations_at_any_element(dtype):
    lora = layer(96, 256, torch.float32)
    x = torch.randn(6 * 256 + 3, device="cuda").to(dtype)[3:].view(6, 256)
    assert x.is_contiguous() and x.data_ptr() % 16 != 0
    assert torch.equal(lora(x), lora(x.clone()))


def test_strided_and_expanded_gradients():
    lora = layer(96, 256, torch.float32)
    x = torch.randn(6, 256, device="cuda", requires_grad=True)
    want, = torch.autograd.grad(lora(x), x, torch.ones(6, 96, device="cuda"))
    got, = torch.autograd.grad(lora(x).sum(), x)
    assert torch.equal(got, want)
    dy = torch.randn(96, 6, device="cuda")
    assert torch.equal(torch.autograd.grad(lora(x), x, dy.t())[0], torch.autograd.grad(lora(x), x, dy.t().contiguous())[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_parameters_that_are_views_of_one_vector(dtype):
    """Parameters in one vector, as optimizers that flatten them leave them, behind one of an odd length."""
    lora = layer(101, 256, dtype)
    x = torch.randn(6, 256, device="cuda").to(dtype)
    dy = torch.randn(6, 101, device="cuda").to(dtype)
    want = lora(x)
    wanted = torch.autograd.grad(want, (lora.a, lora.b), dy)
    odd = torch.zeros(3, device="cuda", dtype=dtype)
    vector = torch.nn.utils.parameters_to_vector([odd, lora.a, lora.b]).detach().clone()
    torch.nn.utils.vector_to_parameters(vector, [odd, lora.a, lora.b])
    assert lora.a.data_ptr() % 16 != 0
    got = lora(x)
    assert torch.equal(got, want)
    assert all(torch.equal(g, w) for g, w in zip(torch.autograd.grad(got, (lora.a, lora.b), dy), wanted))
