"""The products by expert against the oracle: ragged and empty experts, rows
that no expert owns, every kernel of the choice.

Exact construction: integer data whose every partial sum is exact in float32
(MXFP4 as in test_gpu_mxfp4; INT4: x integer in -8..8, scales 2^-3..1, so
products are multiples of 2^-3 and sums stay below 2^21), so a result has to
equal the oracle's rounding.  Real data: K additions off by 2^-23 of at most
S = sum |x w| each, one more rounding a group where the scale is applied, and
the result's own rounding.
"""
import numpy as np
import pytest
import torch

import oracle.mxfp4_oracle as MX
import oracle.w4_oracle as O
from tests.gpu_util import Canary, to_dev, to_host, y_as_f64
from tests.test_gpu_mxfp4 import bound, exact_operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import dequant_gemm_quantize_amd as m
    m.load()
    return m


# rows of each expert, rows before the first and behind the last
SPLITS = {
    "one": ([1], 0, 0),
    "few": ([0, 2, 0, 1, 1, 0], 0, 0),
    "empty": ([0, 0, 0], 0, 5),
    "padded": ([3, 0, 17, 16, 40], 4, 7),
    "many": ([1 if i % 3 == 0 else 0 for i in range(150)], 0, 2),
    "skewed": ([0] * 15 + [37] + [0] * 5, 1, 2),
    "wide": ([70, 0, 129, 33, 1, 256], 1, 30),
    "large": ([300, 257, 0, 511, 65], 0, 9),
}
# with these the tiles fill several rounds of the chip
MANY = {"two": ([600, 500], 0, 3), "uneven": ([1000, 1, 129, 0, 700, 256], 2, 0), "dozen": ([100] * 7 + [0, 130, 260], 0, 0)}


def offsets_of(split):
    sizes, before, behind = {**SPLITS, **MANY}[split]
    off = np.concatenate([[0], np.cumsum(sizes)]) + before
    return off.astype(np.int32), int(off[-1]) + behind


def dtype_of(out):
    return torch.float32 if out == "f32" else torch.bfloat16


def filled(t, n, dt):
    c = Canary((t, n), dt)
    c.tensor.fill_(-7.0)
    return c


MX_SHAPES = [(33, 96), (64, 512), (129, 256), (300, 1152), (256, 2048)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("n,k", MX_SHAPES)
@pytest.mark.parametrize("split", sorted(SPLITS))
def test_mxfp4_exact(w4, split, n, k, out):
    off, t = offsets_of(split)
    e = len(off) - 1
    rng = np.random.default_rng(n + k + t)
    x, w = exact_operand(rng, t, k), exact_operand(rng, e * n, k)
    wq, ws = w[0].reshape(e, n, -1), w[1].reshape(e, n, -1)
    c = filled(t, n, dtype_of(out))
    w4.mxfp4_grouped_matmul(to_dev(x[0], "u8"), to_dev(x[1], "u8"), to_dev32(off), to_dev(wq, "u8"), to_dev(ws, "u8"),
                            out=c.tensor)
    c.check()
    want, _ = MX.grouped(MX.values(*x), MX.values(wq, ws), off, np.full((t, n), -7.0))
    assert torch.equal(c.tensor.cpu(), torch.from_numpy(want).to(dtype_of(out)))


def to_dev32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def int4_exact(rng, t, e, n, k, g):
    x = rng.integers(-8, 9, (t, k)).astype(np.float32)
    code = rng.integers(0, 16, (e, n, k)).astype(np.uint8)
    s = np.ldexp(1.0, rng.integers(-3, 1, (e, n, k // g))).astype(np.float32)
    z = rng.integers(0, 16, (e, n, k // g)).astype(np.float32)
    w = (code.astype(np.float64) - np.repeat(z, g, -1)) * np.repeat(s, g, -1)
    return x, MX.pack(code), s, z, w


W4_SHAPES = [(33, 96, 32), (64, 512, 128), (129, 256, 64), (300, 1152, 128), (100, 672, 96), (256, 2048, 256),
             (70, 1024, 1024)]


@pytest.mark.parametrize("xd,sz,out", [("bf16", "f16", "bf16"), ("bf16", "f32", "f32"), ("f32", "f16", "f32"),
                                       ("f32", "f32", "bf16")])
@pytest.mark.parametrize("n,k,g", W4_SHAPES)
@pytest.mark.parametrize("split", sorted(SPLITS))
def test_w4a16_exact(w4, split, n, k, g, xd, sz, out):
    off, t = offsets_of(split)
    rng = np.random.default_rng(n + k + t + g)
    x, p, s, z, w = int4_exact(rng, t, len(off) - 1, n, k, g)
    xt = to_dev(x, "f32").to(torch.bfloat16 if xd == "bf16" else torch.float32)
    c = filled(t, n, dtype_of(out))
    w4.w4a16_grouped_matmul(xt, to_dev32(off), to_dev(p, "u8"), to_dev(s, sz), to_dev(z, sz), g, out=c.tensor)
    c.check()
    want, _ = MX.grouped(x.astype(np.float64), w, off, np.full((t, n), -7.0))
    assert torch.equal(c.tensor.cpu(), torch.from_numpy(want).to(dtype_of(out)))


# few rows and many weight rows: workgroups of 1, 2, 4 and 6 blocks of 16 weight rows
@pytest.mark.parametrize("n,k,g", [(4001, 512, 128), (8001, 640, 128), (11001, 1152, 384), (17003, 4480, 128),
                                   (9001, 544, 32), (4001, 2240, 64), (8001, 416, 32), (11001, 960, 64)])
@pytest.mark.parametrize("split", ["one", "few"])
def test_exact_many_weight_rows(w4, split, n, k, g):
    test_mxfp4_exact(w4, split, n, k, "f32")
    test_w4a16_exact(w4, split, n, k, g, "bf16", "f16", "bf16")
    test_w4a16_exact(w4, split, n, k, g, "f32", "f32", "f32")


# whole tiles, halves and both, of every size
@pytest.mark.parametrize("n,k", [(1400, 256), (5001, 128), (8000, 384), (14000, 128)])
@pytest.mark.parametrize("split", sorted(MANY))
def test_mxfp4_exact_many_tiles(w4, split, n, k):
    test_mxfp4_exact(w4, split, n, k, "f32")


@pytest.mark.parametrize("n,k,g", [(1400, 192, 64), (7168, 128, 128), (14001, 128, 32)])
@pytest.mark.parametrize("split", sorted(MANY))
def test_w4a16_exact_many_tiles(w4, split, n, k, g):
    test_w4a16_exact(w4, split, n, k, g, "bf16", "f16", "bf16")


@pytest.mark.parametrize("sz", ["f16", "f32"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("split,n,k,g", [("few", 500, 4096, 128), ("padded", 260, 2048, 64), ("large", 300, 2048, 128),
                                         ("wide", 200, 1120, 32)])
def test_w4a16_real(w4, split, n, k, g, out, sz):
    off, t = offsets_of(split)
    e = len(off) - 1
    rng = np.random.default_rng(n + k)
    xt = to_dev(rng.normal(0, 1, (t, k)).astype(np.float32), "f32").to(torch.bfloat16)
    wt = to_dev(rng.normal(0, 0.02, (e * n, k)).astype(np.float32), "f32")
    p, s, z = w4.quantize_pack_int4(wt, g, torch.float16 if sz == "f16" else torch.float32)
    ng = k // g
    y = w4.w4a16_grouped_matmul(xt, to_dev32(off), p.view(e, n, k // 2), s.view(e, n, ng), z.view(e, n, ng), g,
                                out=torch.zeros((t, n), dtype=dtype_of(out), device="cuda"))
    w = O.dequant_f64(to_host(p), to_host(s), to_host(z), g).reshape(e, n, k)
    x = xt.double().cpu().numpy()
    ref, xw = MX.grouped(x, w, off, np.zeros((t, n)))
    # Few rows an expert: the library multiplies x by 16 + q and takes
    # (16 + zp) times the group's sum of x off again, so its sums are of terms
    # up to |x| (16 + 15) s, twice, not |x w|: additions and the scale's
    # rounding are off by 2^-23 of those sums.
    s64 = np.repeat(to_host(s).astype(np.float64).reshape(e, n, ng), g, -1)
    _, mag = MX.grouped(x, 62 * s64, off, np.zeros((t, n)))
    # Many rows an expert: the weight is rounded to bf16, off by 2^-8 |w| at
    # most, for bf16 results; for float32 ones what that rounding lacks is
    # rounded in turn and added, which leaves 2^-8 2^-8 |w|, with float32
    # scales too.  The weight itself, fma(q, s, -zp s), is off by two float32
    # roundings of values up to 15 s: with x, 2^-23 of terms that mag has.
    # Each adds its part of sum |x w| to the result's error before its rounding.
    lost = xw * (2.0 ** -16 if out == "f32" else 2.0 ** -8 * (1 + 2.0 ** -8))
    assert (np.abs(y_as_f64(y) - ref) <= bound(ref, mag, k + 2 * ng, out) + lost).all()



@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("split,n,k,g", [("few", 500, 4096, 128), ("padded", 260, 2048, 64), ("wide", 200, 1120, 32),
                                         ("one", 9000, 1280, 256)])
def test_w4a16_real_float32_x(w4, split, n, k, g, out):
    """float32 x, of which the library adds three parts: 3 K additions in place of K in test_w4a16_real's bound,
    and no rounded weight.  Values from 2^-60 to 2^60 side by side in different rows."""
    off, t = offsets_of(split)
    e, ng = len(off) - 1, k // g
    rng = np.random.default_rng(n + k)
    x = (rng.normal(0, 1, (t, k)) * np.ldexp(1.0, rng.integers(-60, 61, (t, 1)))).astype(np.float32)
    p, s, z = w4.quantize_pack_int4(to_dev(rng.normal(0, 0.02, (e * n, k)).astype(np.float32), "f32"), g)
    y = w4.w4a16_grouped_matmul(to_dev(x, "f32"), to_dev32(off), p.view(e, n, k // 2), s.view(e, n, ng),
                                z.view(e, n, ng), g, out=torch.zeros((t, n), dtype=dtype_of(out), device="cuda"))
    w = O.dequant_f64(to_host(p), to_host(s), to_host(z), g).reshape(e, n, k)
    x = x.astype(np.float64)
    ref, _ = MX.grouped(x, w, off, np.zeros((t, n)))
    s64 = np.repeat(to_host(s).astype(np.float64).reshape(e, n, ng), g, -1)
    _, mag = MX.grouped(x, 62 * s64, off, np.zeros((t, n)))
    assert (np.abs(y_as_f64(y) - ref) <= bound(ref, mag, 3 * k + 2 * ng, out)).all()


@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
@pytest.mark.parametrize("split", ["few", "padded", "wide"])
def test_experts_layer(w4, fmt, split):
    """Up, activation, down through QuantizedExperts, against the oracle step by step."""
    off, t = offsets_of(split)
    e = len(off) - 1
    rng = np.random.default_rng(t)
    up = w4.QuantizedExperts.from_weight(to_dev(rng.normal(0, 0.05, (e, 160, 256)).astype(np.float32), "f32"), fmt=fmt,
                                         group_size=64)
    down = w4.QuantizedExperts.from_weight(to_dev(rng.normal(0, 0.05, (e, 96, 160)).astype(np.float32), "f32"), fmt=fmt,
                                           group_size=32)
    x = torch.randn((t, 256), device="cuda").to(torch.bfloat16)
    offd = to_dev32(off)
    out = torch.zeros((t, 96), dtype=torch.float32, device="cuda")
    h = torch.zeros((t, 160), dtype=torch.bfloat16, device="cuda")
    up(x, offd, out=h)
    a = torch.nn.functional.silu(h.float()).to(torch.bfloat16)
    down(a, offd, out=out)
    for layer, xin, y, k, fin in ((up, x, h, 256, "bf16"), (down, a, out, 160, "f32")):
        wd = layer.dequantize(torch.float32).double().cpu().numpy()
        if fmt == "mxfp4":
            q = w4.quantize_mxfp4(xin)
            xv = MX.values(to_host(q[0]), to_host(q[1]))
            ref, mag = MX.grouped(xv, wd, off, np.zeros(tuple(y.shape)))
            lost = 0.0
        else:
            xv = xin.double().cpu().numpy()
            ref, xw = MX.grouped(xv, wd, off, np.zeros(tuple(y.shape)))
            s64 = np.repeat(layer.scales.double().cpu().numpy(), layer.group_size, -1)
            _, mag = MX.grouped(xv, 62 * s64, off, np.zeros(tuple(y.shape)))
            # dequantize() rounds the weight to float32 once
            mag = mag * 1.01
            # with many rows an expert the product rounds the weight too (test_w4a16_real)
            lost = xw * (2.0 ** -16 if fin == "f32" else 2.0 ** -8 * (1 + 2.0 ** -8))
        assert (np.abs(y_as_f64(y) - ref) <= bound(ref, mag, 2 * k, fin) + lost).all()


@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
def test_graph_replays_with_other_offsets(w4, fmt):
    """One captured graph, offsets changed in place between replays: every replay equals the eager call."""
    rng = np.random.default_rng(8)
    t, e, n, k, g = 600, 6, 200, 512, 128
    x = torch.randn((t, k), device="cuda").to(torch.bfloat16)
    layer = w4.QuantizedExperts.from_weight(torch.randn((e, n, k), device="cuda") * 0.05, fmt=fmt, group_size=g)
    offd = to_dev32(np.zeros(e + 1))
    y = torch.zeros((t, n), dtype=torch.float32, device="cuda")
    layer(x, offd, out=y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        layer(x, offd, out=y)
    torch.cuda.current_stream().wait_stream(side)
    for cuts in ([0, 0, 0, 0, 0, 0, 0], [0, 600, 600, 600, 600, 600, 600], [5, 6, 100, 100, 350, 351, 590],
                 [0, 100, 200, 300, 400, 500, 600]):
        offd.copy_(to_dev32(np.array(cuts)))
        want = torch.full((t, n), 3.0, device="cuda")
        layer(x, offd, out=want)
        y.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), cuts


@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
def test_two_streams_at_once(w4, fmt):
    t, e, n, k = 300, 4, 256, 1024
    layer = w4.QuantizedExperts.from_weight(torch.randn((e, n, k), device="cuda") * 0.05, fmt=fmt)
    xs = [torch.randn((t, k), device="cuda").to(torch.bfloat16) for _ in range(2)]
    offs = [to_dev32(np.array(c)) for c in ([0, 10, 150, 150, 300], [0, 200, 200, 299, 300])]
    want = [layer(x, o) for x, o in zip(xs, offs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for x, o, s in zip(xs, offs, streams):
            with torch.cuda.stream(s):
                got.append(layer(x, o))
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % 2])


@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
@pytest.mark.parametrize("cuts", [[0, 500, 100, 300], [-5, 20, 40, 1 << 30], [300, 200, 100, 0], [7, 7, 7, 7]])
def test_offsets_out_of_order_stay_in_bounds(w4, fmt, cuts):
    """Offsets outside the contract: whatever is written lies inside y (the kernels clamp every offset to 0..T)."""
    t, e, n, k = 300, 3, 130, 256
    layer = w4.QuantizedExperts.from_weight(torch.randn((e, n, k), device="cuda") * 0.05, fmt=fmt)
    c = filled(t, n, torch.float32)
    layer(torch.randn((t, k), device="cuda"), to_dev32(np.array(cuts)), out=c.tensor)
    c.check()
    assert torch.isfinite(c.tensor).all()


@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
def test_last_expert_of_many_gigabytes(w4, fmt, rows):
    """Codes of 5 GB: the last expert's rows equal the same call with that expert alone, and the dense product.
    x is -1, 0 or 1 and weights are multiples of 2^-3 up to 15: sums below 2^19, exact in any order."""
    e, n, k, g = 20, 16384, 32768, 128
    gen = torch.Generator(device="cuda").manual_seed(9)
    packed = torch.randint(0, 256, (e, n, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
    off = torch.full((e + 1,), 0, dtype=torch.int32, device="cuda")
    off[e] = rows
    alone = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    x = torch.randint(-1, 2, (rows, k), device="cuda", generator=gen).to(torch.bfloat16)
    if fmt == "mxfp4":
        scales = torch.randint(126, 129, (e, n, k // 32), dtype=torch.uint8, device="cuda", generator=gen)
        xq = w4.quantize_mxfp4(x)
        y = w4.mxfp4_grouped_matmul(*xq, off, packed, scales)
        want = w4.mxfp4_grouped_matmul(*xq, alone, packed[-1:], scales[-1:])
        dense = w4.mxfp4_matmul(*xq, packed[-1], scales[-1])
    else:
        scales = torch.randint(0, 4, (e, n, k // g), device="cuda", generator=gen)
        scales = (0.125 * 2.0 ** scales).to(torch.float16)
        zeros = torch.randint(0, 16, (e, n, k // g), device="cuda", generator=gen).to(torch.float16)
        y = w4.w4a16_grouped_matmul(x, off, packed, scales, zeros, g)
        want = w4.w4a16_grouped_matmul(x, alone, packed[-1:], scales[-1:], zeros[-1:], g)
        dense = w4.w4a16_matmul(x, packed[-1], scales[-1], zeros[-1], g)
    assert torch.equal(y, want) and torch.equal(y, dense)
    assert y.float().abs().max() > 0
