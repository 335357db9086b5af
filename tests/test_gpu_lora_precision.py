"""The product with adapters and the transposed one keep their weights: no rounding of (q - zp) s before the product, with few rows or many,
for either type of the result.  The cases and what they may be off are in lora_precision_cases.py; the CPU tests of
test_lora_precision_host.py show that they tell rounded weights."""
import pytest
import torch

import dequant_gemm_quantize_amd as w4
from tests import lora_precision_cases as P
from tests.gpu_util import Canary

pytestmark = pytest.mark.gpu

OUT = {"bf16": torch.bfloat16, "f32": torch.float32}


def weight(c):
    return c["packed"], c["scales"], c["zeros"], c["g"]


def adapter(c, dt):
    return c["a"].to(dt), c["b"].to(dt), c["scaling"], c["offsets"], c["which"]


@pytest.mark.parametrize("sz", ["f16", "f32"])
@pytest.mark.parametrize("out", sorted(OUT))
@pytest.mark.parametrize("shape", P.FORWARD, ids=lambda s: "x".join(map(str, s)))
def test_forward(shape, out, sz):
    c = P.case(*shape, sz, "cuda", sum(shape))
    y = Canary((c["m"], c["n"]), OUT[out])
    w4.w4a16_lora_matmul(c["x"].bfloat16(), *weight(c), *adapter(c, torch.bfloat16), out=y.tensor)
    y.check()
    want = P.forward(c, c["dense"])
    if sz == "f16":
        assert torch.equal(y.tensor, want.to(OUT[out]))
    else:
        assert ((y.tensor.double() - want).abs() <= P.allowance(c, False, OUT[out], want)).all()


@pytest.mark.parametrize("g", [32, 64, 128])
def test_forward_rows_beside_others(g):
    """A row's result is the same to float32's last bits whether it comes alone or with many: bf16 results differ only
    where the exact one lies between two bf16 values and the float32 ones fall on either side."""
    gen = torch.Generator(device="cuda").manual_seed(g)
    m, n, k = 300, 2056, 4096
    x = torch.randn((m, k), generator=gen, device="cuda").bfloat16()
    packed, scales, zeros = w4.quantize_pack_int4(torch.randn((n, k), generator=gen, device="cuda") * 0.02, g)
    ad = (torch.randn((1, 8, k), generator=gen, device="cuda") * k ** -0.5, torch.randn((1, n, 8), generator=gen, device="cuda") * 0.02,
          torch.ones(1, device="cuda"))
    zero = torch.zeros((1,), dtype=torch.int32, device="cuda")
    ends = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    many = w4.w4a16_lora_matmul(x, packed, scales, zeros, g, *ad, ends * m, zero)[-1]
    alone = w4.w4a16_lora_matmul(x[-1:], packed, scales, zeros, g, *ad, ends, zero)[0]
    # half a step of bf16 is 2^-9 of y; the float32 sums differ by about 2^-20 of it, so ties split in far below 2% of cases
    assert (many != alone).double().mean().item() <= 0.02


@pytest.mark.parametrize("sz", ["f16", "f32"])
@pytest.mark.parametrize("out", sorted(OUT))
@pytest.mark.parametrize("shape", P.BACK, ids=lambda s: "x".join(map(str, s)))
def test_back(shape, out, sz):
    c = P.case(*shape, sz, "cuda", sum(shape))
    want = P.back(c, c["dense"])
    plain = c["dy"].double() @ c["dense"]
    for adapters, exact in ((True, want), (False, plain)):
        dx = Canary((c["m"], c["k"]), OUT[out])
        if adapters:
            w4.w4a16_lora_matmul_t(c["dy"].bfloat16(), *weight(c), *adapter(c, torch.bfloat16), out=dx.tensor)
        else:
            w4.w4a16_matmul_t(c["dy"].bfloat16(), *weight(c), out=dx.tensor)
        dx.check()
        if sz == "f16":
            assert torch.equal(dx.tensor, exact.to(OUT[out]))
        else:
            assert ((dx.tensor.double() - exact).abs() <= P.allowance(c, True, OUT[out], exact)).all()
