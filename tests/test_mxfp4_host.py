"""CPU checks of the MXFP4 and by-expert entry points: the oracle's pins, the
C ABI's refusals before any HIP call, and the binding's refusals."""
import os

import numpy as np
import pytest
import torch

import oracle.mxfp4_oracle as MX

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "dequant_gemm_quantize_amd", "libw4.so")
built = pytest.mark.skipif(not os.path.exists(LIB), reason="libw4.so not built")


@pytest.fixture(scope="module")
def lib():
    import dequant_gemm_quantize_amd as w4
    return w4.load()


def test_oracle_rounds_to_the_nearest_value():
    """Against a search over all values: the nearest, the even code on a tie; the error is at most half a step."""
    rng = np.random.default_rng(0)
    w = rng.normal(0, 1, (200, 32)).astype(np.float32)
    w[:, 1] = np.arange(200) / 16.0
    code, byte = MX.quantize(w)
    for r in range(200):
        e = int(byte[r, 0]) - 127
        assert e == int(np.floor(np.log2(np.abs(w[r]).max()))) - 2
        for c in range(32):
            v = abs(float(w[r, c])) / 2.0 ** e
            d = np.abs(MX.E2M1 - v)
            best = np.flatnonzero(d == d.min())
            want = best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1]
            assert code[r, c] & 7 == want, (v, code[r, c])
            assert (code[r, c] >= 8) == np.signbit(w[r, c])


def test_oracle_special_blocks():
    w = np.zeros((1, 128), np.float32)
    w[0, 33], w[0, 64], w[0, 96] = np.float32(2.0 ** -149), np.inf, 6.0
    code, byte = MX.quantize(w)
    assert byte.tolist() == [[0, 0, 255, 127]]
    assert code[0, 96] == 7 and not code[0, :96].any()
    v = MX.values(MX.pack(code), byte)
    assert np.isnan(v[0, 64:96]).all() and v[0, 96] == 6.0


A, U = 0x10000, 0x10002  # aligned / misaligned to 4 bytes; never dereferenced
H = 0x10004              # aligned to 4 bytes, not 16


def err(lib):
    return lib.w4_last_error().decode()


@built
@pytest.mark.parametrize("args,msg", [
    ((A, 2, 4, 100, A, A, None), "k = 100 is not a multiple"),
    ((A, 2, 4, 0, A, A, None), "k = 0"),
    ((A, 2, -1, 32, A, A, None), "n = -1"),
    ((A, 1, 4, 32, A, A, None), "w dtype"),
    ((None, 2, 4, 32, A, A, None), "w is NULL"),
    ((H, 2, 4, 32, A, A, None), "w is not 16-byte aligned"),
    ((A, 2, 4, 32, A, U, None), "scales is not 4-byte aligned"),
    ((A, 2, 1 << 30, 1 << 20, A, A, None), "too large"),
])
def test_quantize_rejects(lib, args, msg):
    assert lib.quantize_mxfp4(*args) == -1
    assert msg in err(lib) and err(lib).startswith("quantize_mxfp4:"), err(lib)


@built
@pytest.mark.parametrize("args,msg", [
    ((A, A, 4, 48, A, 2, None), "k = 48"),
    ((A, A, 4, 64, A, 3, None), "out dtype"),
    ((A, A, 4, 64, None, 2, None), "w_out is NULL"),
])
def test_dequant_rejects(lib, args, msg):
    assert lib.dequant_mxfp4(*args) == -1
    assert msg in err(lib), err(lib)


@built
@pytest.mark.parametrize("args,msg", [
    ((A, A, 3, 80, A, A, 5, A, 2, None), "k = 80"),
    ((A, A, -3, 64, A, A, 5, A, 2, None), "m = -3"),
    ((A, A, 3, 64, A, A, 5, A, 1, None), "y dtype"),
    ((A, None, 3, 64, A, A, 5, A, 2, None), "xs is NULL"),
    ((A, U, 3, 64, A, A, 5, A, 2, None), "xs is not 4-byte"),
    ((A, A, 3, 64, H, A, 5, A, 2, None), "packed is not 16-byte"),
    ((A, A, 3, 64, A, A, 5, H, 2, None), "y is not 16-byte"),
    ((A, A, 1 << 30, 64, A, A, 128, A, 2, None), "m * n is too large"),
])
def test_matmul_rejects(lib, args, msg):
    assert lib.mxfp4_matmul(*args) == -1
    assert msg in err(lib), err(lib)


GROUPED = [
    (dict(t=-1), "m = -1"), (dict(t=(1 << 24) + 1), "at most 16777216"), (dict(e=-1), "experts = -1"),
    (dict(e=65537), "experts = 65537"), (dict(k=72), "k = 72"), (dict(off=None), "offsets is NULL"),
    (dict(off=U), "offsets is not 4-byte"), (dict(x=H), "is not 16-byte"), (dict(yd=1), "y dtype"),
    (dict(e=65536, n=1 << 15, k=64), "experts * n * k"), (dict(y=None), "y is NULL"),
]


@built
@pytest.mark.parametrize("change,msg", GROUPED)
def test_grouped_rejects(lib, change, msg):
    d = dict(x=A, t=4, k=64, off=A, e=3, n=5, y=A, yd=2, **{}) | change
    assert lib.mxfp4_grouped_matmul(d["x"], A, d["t"], d["k"], d["off"], d["e"], A, A, d["n"], d["y"], d["yd"], None) == -1
    assert msg in err(lib), err(lib)
    assert lib.w4a16_grouped_matmul(d["x"], 2, d["t"], d["k"], d["off"], d["e"], A, A, A, 1, d["n"], 32, d["y"], d["yd"],
                                    None) == -1
    assert msg in err(lib), err(lib)


@built
@pytest.mark.parametrize("args,msg", [((1, 1, 32), "x dtype"), ((2, 2, 32), "scale dtype"), ((2, 1, 48), "multiple of 32"),
                                      ((2, 1, 128), "not a multiple of group_size")])
def test_w4a16_grouped_rejects(lib, args, msg):
    xd, sz, g = args
    assert lib.w4a16_grouped_matmul(A, xd, 4, 64, A, 3, A, A, A, sz, 5, g, A, 2, None) == -1
    assert msg in err(lib), err(lib)


@built
def test_empty_calls(lib):
    assert lib.quantize_mxfp4(None, 2, 0, 64, None, None, None) == 0
    assert lib.dequant_mxfp4(None, None, 0, 64, None, 2, None) == 0
    assert lib.mxfp4_matmul(None, None, 0, 64, None, None, 5, None, 2, None) == 0
    assert lib.mxfp4_matmul(None, None, 5, 64, None, None, 0, None, 2, None) == 0
    for t, e, n in ((0, 3, 5), (4, 0, 5), (4, 3, 0)):
        assert lib.mxfp4_grouped_matmul(None, None, t, 64, None, e, None, None, n, None, 2, None) == 0
        assert lib.w4a16_grouped_matmul(None, 2, t, 64, None, e, None, None, None, 1, n, 32, None, 2, None) == 0


# ---- the binding -----------------------------------------------------------------
def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


OFF = torch.zeros(4, dtype=torch.int32)


@built
@pytest.mark.parametrize("call,msg", [
    (lambda w: w.quantize_mxfp4(torch.zeros(2, 48)), "multiple of 32"),
    (lambda w: w.quantize_mxfp4(torch.zeros(64)), "2-D"),
    (lambda w: w.quantize_mxfp4(torch.zeros(2, 64, dtype=torch.float16)), "dtype"),
    (lambda w: w.quantize_mxfp4(torch.zeros(2, 64), out=(u8(2, 32), u8(2, 3))), "scales has shape"),
    (lambda w: w.quantize_mxfp4(torch.zeros(2, 64)), "GPU only"),
    (lambda w: w.dequant_mxfp4(u8(2, 32), u8(2, 1)), "scales has shape"),
    (lambda w: w.dequant_mxfp4(u8(2, 32), u8(2, 2), out_dtype=torch.float64), "unsupported dtype"),
    (lambda w: w.dequant_mxfp4(u8(2, 32), u8(2, 2)), "GPU only"),
    (lambda w: w.mxfp4_matmul(u8(2, 32), u8(2, 2), u8(3, 16), u8(3, 1)), "columns of codes"),
    (lambda w: w.mxfp4_matmul(u8(2, 32), u8(2, 2), u8(3, 32).int(), u8(3, 2)), "dtype"),
    (lambda w: w.mxfp4_matmul(u8(2, 32), u8(2, 2), u8(3, 32), u8(3, 2)), "GPU only"),
    (lambda w: w.mxfp4_grouped_matmul(u8(2, 32), u8(2, 2), OFF, u8(3, 5, 16), u8(3, 5, 1)), "columns of codes"),
    (lambda w: w.mxfp4_grouped_matmul(u8(2, 32), u8(2, 2), OFF, u8(4, 5, 32), u8(4, 5, 2)), "offsets has shape"),
    (lambda w: w.mxfp4_grouped_matmul(u8(2, 32), u8(2, 2), OFF.long(), u8(3, 5, 32), u8(3, 5, 2)), "offsets has dtype"),
    (lambda w: w.mxfp4_grouped_matmul(u8(2, 32), u8(2, 2), OFF, u8(5, 32), u8(5, 2)), "3-D"),
    (lambda w: w.mxfp4_grouped_matmul(u8(2, 32), u8(2, 2), OFF, u8(3, 5, 32), u8(3, 5, 2)), "GPU only"),
    (lambda w: w.w4a16_grouped_matmul(torch.zeros(2, 64), OFF, u8(3, 5, 32), torch.ones(3, 5, 3), torch.ones(3, 5, 2), 32),
     "scales has shape"),
    (lambda w: w.w4a16_grouped_matmul(torch.zeros(2, 64), OFF, u8(3, 5, 32), torch.ones(3, 5, 2), torch.ones(3, 5, 2).half(),
                                      32), "zeros has dtype"),
    (lambda w: w.w4a16_grouped_matmul(torch.zeros(2, 64).half(), OFF, u8(3, 5, 32), torch.ones(3, 5, 2),
                                      torch.ones(3, 5, 2), 32), "dtype"),
    (lambda w: w.w4a16_grouped_matmul(torch.zeros(2, 64), OFF, u8(3, 5, 32), torch.ones(3, 5, 2), torch.ones(3, 5, 2), 32),
     "GPU only"),
])
def test_binding_refuses(call, msg):
    import dequant_gemm_quantize_amd as w4
    with pytest.raises(ValueError, match=msg):
        call(w4)


@built
def test_layers_refuse():
    import dequant_gemm_quantize_amd as w4
    with pytest.raises(ValueError, match="multiple of 32"):
        w4.MXFP4Linear(48, 8)
    with pytest.raises(ValueError, match="bias"):
        w4.MXFP4Linear.from_linear(torch.nn.Linear(64, 8))
    with pytest.raises(ValueError, match="fmt"):
        w4.QuantizedExperts(2, 64, 8, fmt="int3")
    with pytest.raises(ValueError, match="multiple"):
        w4.QuantizedExperts(2, 96, 8, fmt="int4", group_size=64)
    with pytest.raises(ValueError, match=r"\[experts, out, in\]"):
        w4.QuantizedExperts.from_weight(torch.zeros(8, 64))
