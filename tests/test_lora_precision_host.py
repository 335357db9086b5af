"""CPU checks of lora_precision_cases: a product whose weights are rounded to bf16 fails the criteria that the GPU tests
apply, weights in two bf16 parts fail those of a float32 result of float32 scales, and exact ones pass."""
import pytest
import torch

from tests import lora_precision_cases as P

SHAPES = [(24, 130, 512, 128), (24, 70, 320, 64), (16, 66, 192, 96)]


def results(shape, sz, transposed, model):
    c = P.case(*shape, sz, "cpu", sum(shape))
    run = P.back if transposed else P.forward
    return c, run(c, c["dense"]), run(c, model(c["dense"]))


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_half_scales_tell_rounded_weights(shape, transposed):
    c, want, got = results(shape, "f16", transposed, P.bf16)
    assert torch.equal(want * 2 ** 13, (want * 2 ** 13).round()) and want.abs().max() < 2 ** 9
    for dt in (torch.float32, torch.bfloat16):
        assert (got.to(dt) != want.to(dt))[:c["m"] // 2].double().mean() > 0.05
    assert torch.equal(results(shape, "f16", transposed, P.in_two)[2], want)  # two parts hold 11 + 4 bits


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_float_scales_tell_rounded_weights(shape, transposed):
    for model, dt, least in ((P.bf16, torch.float32, 0.9), (P.in_two, torch.float32, 0.2), (P.bf16, torch.bfloat16, 0.05)):
        c, want, got = results(shape, "f32", transposed, model)
        off = (got.to(dt).double() - want).abs() > P.allowance(c, transposed, dt, want)
        assert off[:c["m"] // 2].double().mean() > least, (model, dt)


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_exact_weights_pass(shape, transposed):
    for dt in (torch.float32, torch.bfloat16):
        c, want, _ = results(shape, "f32", transposed, P.bf16)
        assert ((want.to(dt).double() - want).abs() <= P.allowance(c, transposed, dt, want)).all()
    two = results(shape, "f32", True, P.in_two)
    assert ((two[2].bfloat16().double() - two[1]).abs() <= P.allowance(two[0], True, torch.bfloat16, two[1])).all()
