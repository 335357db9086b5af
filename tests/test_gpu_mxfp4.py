"""MXFP4 on the GPU: quantize and dequantize bit for bit against the oracle,
the product against it in two ways.

* exact: scale bytes 126..128, so that every product is a multiple of 2^-4 and
  every partial sum stays below 2^20: each float32 sum is exact in any order,
  and a float32 result has to equal the oracle's, a bfloat16 one its rounding.
  A wrong code, scale or row changes it.
* real: normal data.  Products are exact in float32; each of the K additions
  is off by at most 2^-23 of a partial sum that is at most S = sum |x w|, so a
  float32 result is within K 2^-23 S; rounding to bfloat16 adds 2^-8 |y|
  (of the rounded value: 2^-8 (1 + 2^-8) |y| of the exact one).
"""
import numpy as np
import pytest
import torch

import oracle.mxfp4_oracle as MX
import oracle.w4_oracle as O
from tests.gpu_util import Canary, to_dev, to_host, y_as_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import dequant_gemm_quantize_amd as m
    m.load()
    return m


def extremes(rng):
    """Rows over the whole float32 range, every rounding border and its neighbours, zeros and subnormals."""
    rows = [rng.normal(0, 1, (300, 64)) * np.logspace(-45, 37, 300)[:, None]]
    grid = np.arange(-512, 512) / 64.0
    for e in (-127, -126, -60, 0, 119):
        b = np.zeros((1024, 64))
        b[:, 0], b[:, 32], b[:, 1], b[:, 33] = 7.0, -6.0, grid, grid
        up = np.nextafter(grid.astype(np.float32), np.float32(np.inf)).astype(np.float64)
        b[:, 2], b[:, 40] = up, -up
        rows.append(np.ldexp(b, e))
    tiny = np.array([2.0 ** -149, 2.0 ** -127, 2.0 ** -126, 3.4e38, 1.8e38, 0.0, -0.0])
    rows.append(np.repeat(tiny[:, None], 64, 1))
    return np.concatenate(rows).astype(np.float32)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantize_extremes(w4, kind):
    w = extremes(np.random.default_rng(1))
    t = to_dev(w, "f32")
    if kind == "bf16":
        t = t.to(torch.bfloat16)
        w = t.float().cpu().numpy()
    p, s = w4.quantize_mxfp4(t)
    code, byte = MX.quantize(w)
    assert np.array_equal(to_host(s), byte)
    assert np.array_equal(to_host(p), MX.pack(code))


@pytest.mark.parametrize("n,k", [(1, 32), (1, 4096), (3, 96), (257, 160), (64, 11008), (70001, 32)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_quantize_sizes(w4, n, k, kind):
    t = to_dev(np.random.default_rng(n + k).normal(0, 1, (n, k)).astype(np.float32), "f32")
    t = t.to(torch.bfloat16) if kind == "bf16" else t
    p, s = Canary((n, k // 2), torch.uint8), Canary((n, k // 32), torch.uint8)
    w4.quantize_mxfp4(t, out=(p.tensor, s.tensor))
    p.check(), s.check()
    code, byte = MX.quantize(t.float().cpu().numpy())
    assert np.array_equal(to_host(s.tensor), byte)
    assert np.array_equal(to_host(p.tensor), MX.pack(code))


def test_quantize_marks_blocks_that_are_not_finite(w4):
    w = np.random.default_rng(2).normal(0, 1, (4, 128)).astype(np.float32)
    w[0, 5], w[1, 64], w[2, 127], w[3, 0] = np.inf, -np.inf, np.nan, 3e38
    p, s = w4.quantize_mxfp4(to_dev(w, "f32"))
    code, byte = MX.quantize(w)
    assert np.array_equal(to_host(s), byte) and (byte == 255).sum() == 3
    assert np.array_equal(to_host(p), MX.pack(code))
    v = w4.dequant_mxfp4(p, s, out_dtype=torch.float32).cpu().numpy()
    assert np.array_equal(np.isnan(v), np.repeat(byte == 255, 32, axis=1))
    # a product with such a row is NaN there and nowhere else
    one = MX.pack(np.full((5, 128), 2, np.uint8)), np.full((5, 4), 127, np.uint8)
    y = w4.mxfp4_matmul(p, s, to_dev(one[0], "u8"), to_dev(one[1], "u8"), out_dtype=torch.float32).cpu().numpy()
    assert np.isnan(y[:3]).all() and np.isfinite(y[3]).all()


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_dequant_every_code_and_scale(w4, out):
    """All 256 code pairs under all 256 scale bytes."""
    p = np.tile(np.arange(256, dtype=np.uint8).reshape(1, 256), (256, 1))
    s = np.tile(np.arange(256, dtype=np.uint8).reshape(256, 1), (1, 16))
    dt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[out]
    c = Canary((256, 512), dt)
    w4.dequant_mxfp4(to_dev(p, "u8"), to_dev(s, "u8"), out=c.tensor)
    c.check()
    v = torch.from_numpy(MX.values(p, s))
    want = v.to(torch.float32).to(dt)  # the value is exact in float32 or beyond its range
    got = c.tensor.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])


def exact_operand(rng, rows, k):
    code = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    return MX.pack(code), rng.integers(126, 129, (rows, k // 32)).astype(np.uint8)


def dev(op):
    return to_dev(op[0], "u8"), to_dev(op[1], "u8")


SHAPES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (1, 300, 512), (5, 33, 544), (16, 64, 1024), (17, 100, 160),
          (33, 15, 2048), (64, 48, 1152), (65, 129, 256), (80, 64, 672), (100, 257, 128), (129, 300, 384),
          (200, 513, 640), (256, 256, 512), (257, 130, 1664), (300, 1000, 1920), (511, 770, 2048), (700, 260, 896)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_matmul_exact(w4, m, n, k, out):
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    x, w = exact_operand(rng, m, k), exact_operand(rng, n, k)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    c = Canary((m, n), dt)
    w4.mxfp4_matmul(*dev(x), *dev(w), out=c.tensor)
    c.check()
    want = torch.from_numpy(MX.matmul(*x, *w)[0]).to(dt)
    assert torch.equal(c.tensor.cpu(), want)


# Many tiles: 256 x 256 and 256 x 192 ones, whole, in halves and both, with
# and without a last half step of K, rows of y that start anywhere.
@pytest.mark.parametrize("m,n,k", [(2000, 8190, 384), (1500, 4100, 256), (1530, 2999, 640), (2048, 4352, 128),
                                   (1100, 13000, 256), (4200, 4501, 128)])
def test_matmul_exact_many_tiles(w4, m, n, k):
    test_matmul_exact(w4, m, n, k, "f32")
    test_matmul_exact(w4, m, n, k, "bf16")


# Few rows and many weight rows: workgroups of 1, 2, 4 and 6 blocks of 16 weight
# rows, whole slices of K and a partial one, one or two slices a wave.
@pytest.mark.parametrize("m,n,k", [(1, 8001, 544), (16, 11001, 512), (3, 20003, 96), (9, 17000, 1056), (20, 8001, 544),
                                   (32, 11001, 512), (40, 4600, 1024), (130, 4600, 160), (2, 700, 8736)])
def test_matmul_exact_many_weight_rows(w4, m, n, k):
    test_matmul_exact(w4, m, n, k, "f32")
    test_matmul_exact(w4, m, n, k, "bf16")


def bound(y, mag, k, out):
    err = k * 2.0 ** -23 * mag
    return err if out == "f32" else err * (1 + 2.0 ** -8) + 2.0 ** -8 * (1 + 2.0 ** -8) * np.abs(y)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 500, 4096), (7, 300, 11008), (40, 200, 2080), (130, 400, 4096),
                                   (600, 520, 2304)])
def test_matmul_real(w4, m, n, k, out):
    rng = np.random.default_rng(m + n + k)
    x, w = rng.normal(0, 1, (m, k)).astype(np.float32), rng.normal(0, 0.02, (n, k)).astype(np.float32)
    x[:, :: 20] *= 20
    xq, wq = w4.quantize_mxfp4(to_dev(x, "f32")), w4.quantize_mxfp4(to_dev(w, "f32"))
    y = w4.mxfp4_matmul(*xq, *wq, out_dtype=torch.float32 if out == "f32" else torch.bfloat16)
    ref, mag = MX.matmul(*(to_host(t) for t in (*xq, *wq)))
    assert (np.abs(y_as_f64(y) - ref) <= bound(ref, mag, k, out)).all()


@pytest.mark.parametrize("m", [1, 300])
def test_matmul_scales_over_the_whole_range(w4, m):
    """Scale bytes whose sum spans float32's exponents: zero products, huge and tiny blocks side by side."""
    rng = np.random.default_rng(3)
    n, k = 200, 512
    x, w = exact_operand(rng, m, k), exact_operand(rng, n, k)
    xs, ws = x[1].copy(), w[1].copy()
    xs[:, 0], ws[:, 0] = 0, 254       # 2^-127 2^127
    xs[:, 1], ws[:, 1] = 230, 24
    xs[:, 2], ws[:, 2] = 1, 253
    y = w4.mxfp4_matmul(*dev((x[0], xs)), *dev((w[0], ws)), out_dtype=torch.float32)
    # the three blocks' products have byte sum 254: multiples of 2^-2, like the others exact
    assert torch.equal(y.cpu(), torch.from_numpy(MX.matmul(x[0], xs, w[0], ws)[0]).float())


def test_matmul_takes_row_slices(w4):
    """Rows of a larger batch: scale rows of K/32 bytes that start at 4-byte addresses only."""
    rng = np.random.default_rng(4)
    for m, k in ((9, 128), (150, 128), (9, 384), (150, 384)):
        x, w = exact_operand(rng, m + 3, k), exact_operand(rng, 70, k)
        xd, wd = dev(x), dev(w)
        y = w4.mxfp4_matmul(xd[0][3:], xd[1][3:], wd[0], wd[1], out_dtype=torch.float32)
        assert torch.equal(y.cpu(), torch.from_numpy(MX.matmul(x[0][3:], x[1][3:], *w)[0]).float())


def test_layer_chain(w4):
    """Quantize the activations, multiply, quantize the result, multiply: as a model's two linears."""
    rng = np.random.default_rng(5)
    x = rng.normal(0, 1, (37, 512)).astype(np.float32)
    w1, w2 = (rng.normal(0, 0.05, s).astype(np.float32) for s in ((384, 512), (96, 384)))
    model = torch.nn.Sequential(torch.nn.Linear(512, 384, bias=False), torch.nn.Linear(384, 96, bias=False)).cuda()
    with torch.no_grad():
        model[0].weight.copy_(to_dev(w1, "f32"))
        model[1].weight.copy_(to_dev(w2, "f32"))
    w4.replace_linears(model, mode="mxfp4", out_dtype=torch.float32)
    assert [type(l).__name__ for l in model] == ["MXFP4Linear", "MXFP4Linear"]
    y = model(to_dev(x, "f32"))
    h = model[0](to_dev(x, "f32"))
    c, s = MX.quantize(x)
    c1, s1 = MX.quantize(w1)
    ref, mag = MX.matmul(MX.pack(c), s, MX.pack(c1), s1)
    assert (np.abs(y_as_f64(h) - ref) <= bound(ref, mag, 512, "f32")).all()
    c, s = MX.quantize(h.cpu().numpy())
    c2, s2 = MX.quantize(w2)
    ref, mag = MX.matmul(MX.pack(c), s, MX.pack(c2), s2)
    assert (np.abs(y_as_f64(y) - ref) <= bound(ref, mag, 384, "f32")).all()
    assert np.array_equal(model[0].dequantize(torch.float32).cpu().numpy(), MX.values(MX.pack(c1), s1).astype(np.float32))


def test_layer_shapes_and_dtypes(w4):
    w = to_dev(np.random.default_rng(6).normal(0, 0.02, (48, 96)).astype(np.float32), "f32")
    layer = w4.MXFP4Linear.from_weight(w.to(torch.float16))
    y = layer(torch.randn(2, 5, 96, device="cuda", dtype=torch.bfloat16))
    assert tuple(y.shape) == (2, 5, 48) and y.dtype == torch.bfloat16
    assert layer(torch.randn(96, device="cuda")).shape == (48,)
    assert layer(torch.randn(0, 96, device="cuda")).shape == (0, 48)
    with pytest.raises(ValueError, match="features"):
        layer(torch.randn(2, 64, device="cuda"))
