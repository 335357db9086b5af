"""The INT4 product by expert keeps its weights: no rounding of (q - zp) s
before the product, with few rows an expert or many, for either type of y.
The cases and what they may be off are in grouped_cases.py; the CPU tests of
test_grouped_precision_host.py show that they tell rounded weights."""
import numpy as np
import pytest
import torch

import oracle.mxfp4_oracle as MX
import oracle.w4_oracle as O
import tests.grouped_cases as GC
from tests.gpu_util import Canary, to_dev, y_as_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import dequant_gemm_quantize_amd as m
    m.load()
    return m


def product(w4, x, code, s, z, g, off, out, xd="bf16", sz="f16"):
    c = Canary((x.shape[0], code.shape[1]), torch.float32 if out == "f32" else torch.bfloat16)
    c.tensor.fill_(-7.0)
    xt = to_dev(x, "f32").to(torch.bfloat16 if xd == "bf16" else torch.float32)
    w4.w4a16_grouped_matmul(xt, torch.from_numpy(off).cuda(), to_dev(MX.pack(code), "u8"), to_dev(s, sz), to_dev(z, sz), g,
                            out=c.tensor)
    c.check()
    return c.tensor


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,g", GC.SHAPES)
@pytest.mark.parametrize("split", sorted(GC.SPLITS))
def test_half_scales_exact(w4, split, n, k, g, out):
    off, t = GC.offsets_of(split)
    x, code, s, z = GC.sparse_scales_f16(np.random.default_rng(n + k + g + t), t, len(off) - 1, n, k, g)
    y = product(w4, x, code, s, z, g, off, out)
    want = torch.from_numpy(GC.exact(x, GC.weights(code, s, z, g), off, t, n, -7.0)).to(y.dtype)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("n,k,g", GC.SHAPES)
@pytest.mark.parametrize("split", sorted(GC.SPLITS))
def test_float_scales_kept_whole(w4, split, n, k, g):
    off, t = GC.offsets_of(split)
    x, code, s, z = GC.sparse_scales_f32(np.random.default_rng(n + k + g + t), t, len(off) - 1, n, k, g)
    y = product(w4, x, code, s, z, g, off, "f32", sz="f32")
    want = GC.exact(x, GC.weights(code, s, z, g), off, t, n, -7.0)
    assert (np.abs(y_as_f64(y) - want) <= GC.allowance_f32(x, s, g, off)).all()


@pytest.mark.parametrize("g", [32, 64, 128])
def test_rows_beside_others(w4, g):
    """A row's result is the same to float32's last bits whether it comes alone or with many: bf16 y differ only where
    the exact result lies between two bf16 values and the float32 ones fall on either side."""
    rng = np.random.default_rng(g)
    n, k, e = 200, 1024, 2
    x = torch.from_numpy(rng.normal(0, 1, (300, k)).astype(np.float32)).to(torch.bfloat16).cuda()
    layer = w4.QuantizedExperts.from_weight(torch.from_numpy(rng.normal(0, 0.02, (e, n, k)).astype(np.float32)).cuda(),
                                            group_size=g)
    off = torch.tensor([0, 299, 300], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")
    many, alone = layer(x, off)[-1], layer(x[-1:].contiguous(), one)[0]
    w = layer.dequantize(torch.float32)[1].double()
    ref = (w @ x[-1].double())
    # each is off by its bf16 rounding and by float32 errors far below it: K 2^-23 of sums of 62 |x| s at most
    mag = 62 * (layer.scales[1].double().repeat_interleave(g, 1) @ x[-1].double().abs())
    tol = 2.0 ** -8 * (1 + 2.0 ** -8) * ref.abs() + 1.01 * (k + 2 * k // g) * 2.0 ** -23 * mag
    assert ((many.double() - ref).abs() <= tol).all() and ((alone.double() - ref).abs() <= tol).all()
    near = (many != alone).double().mean().item()
    # half a step of bf16 is 2^-9 |y|; the float32 sums differ by about 2^-20 of it, so ties split in far below 2% of cases
    assert near <= 0.02


@pytest.mark.parametrize("sz", ["f16", "f32"])
@pytest.mark.parametrize("n,k,g", GC.SHAPES + [(100, 672, 96), (9001, 256, 128)])
@pytest.mark.parametrize("split", sorted(GC.SPLITS))
def test_wide_float32_x_exact(w4, split, n, k, g, sz):
    """float32 x whose middle and lower bf16 parts count."""
    off, t = GC.offsets_of(split)
    x, code, s, z = GC.wide_x(np.random.default_rng(n + k + g + t), t, len(off) - 1, n, k, g)
    y = product(w4, x, code, s, z, g, off, "f32", xd="f32", sz=sz)
    want = torch.from_numpy(GC.exact(x, GC.weights(code, s, z, g), off, t, n, -7.0)).to(torch.float32)
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("xd", ["f32", "bf16"])
@pytest.mark.parametrize("split,n,k,g", [("few", 500, 4096, 128), ("some", 260, 2048, 64), ("many", 200, 1120, 32),
                                         ("many", 300, 2048, 128), ("most", 130, 1024, 32), ("most", 200, 1280, 256)])
def test_real_data_to_float32(w4, split, n, k, g, xd):
    """Normal data, float32 y, against 64 bits with a bound that grows with the root of K."""
    off, t = GC.offsets_of(split)
    e, ng = len(off) - 1, k // g
    x, wf = GC.real_float_x(np.random.default_rng(n + k), t, e, n, k)
    x = GC.bf16(x) if xd == "bf16" else x
    xt = to_dev(x, "f32").to(torch.bfloat16 if xd == "bf16" else torch.float32)
    p, s, z = w4.quantize_pack_int4(to_dev(wf, "f32"), g)
    y = w4.w4a16_grouped_matmul(xt, torch.from_numpy(off).cuda(), p.view(e, n, k // 2), s.view(e, n, ng), z.view(e, n, ng), g,
                                out=torch.zeros((t, n), dtype=torch.float32, device="cuda"))
    sh = s.float().cpu().numpy().reshape(e, n, ng)
    w = O.dequant_f64(p.cpu().numpy(), s.cpu().numpy(), z.cpu().numpy(), g).reshape(e, n, k)
    assert (np.abs(y_as_f64(y) - GC.exact(x, w, off, t, n)) <= GC.allowance_real(x, sh, g, off)).all()
