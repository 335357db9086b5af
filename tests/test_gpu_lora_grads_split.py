"""lora_grads where the rows are split among workgroups and a second kernel adds their sums: bit for bit on whole numbers,
with exactly the workspace that the size function asks for, at the edges of parts and of the two results."""
import ctypes

import pytest
import torch

import dequant_gemm_quantize_amd as w4
from dequant_gemm_quantize_amd import _lib
from tests import lora_cases as C
from tests.gpu_util import Canary

pytestmark = pytest.mark.gpu

# rows, out, in, rank, bounds, adapters of the segments, number of adapters.  Parts have 64 rows a wave, four waves: two parts
# from 512 rows on.  Ragged n; adapters without rows, with fewer steps of 32 rows than there are waves in all parts, and with rows
# in several segments; ranks of one, two and four blocks of 16.
SHAPES = {
    "two parts": (512, 96, 128, 16, [0, 512], [0], 1),
    "two parts and a row": (513, 101, 160, 8, [0, 513], [0], 1),
    "rows before and behind": (2049, 33, 96, 16, [3, 1000, 2040], [0, 0], 1),
    "an adapter without rows": (2049, 130, 288, 40, [0, 40, 700, 2049], [0, 2, 0], 3),
    "few steps a part": (2100, 70, 256, 64, [0, 33, 2000, 2064, 2100], [1, -1, 0, 1], 2),
    "many small segments": (1600, 64, 64, 24, list(range(0, 1601, 16)), [i % 3 - 1 for i in range(100)], 2),
    "many parts": (9000, 10, 32, 8, [0, 4500, 9000], [1, 0], 2),
    "wide": (1100, 2050, 1024, 16, [0, 600, 1100], [1, 0], 2),
}


def make(name, dy):
    m, n, k, r, bounds, which, l = SHAPES[name]
    c = C.case(m, n, k, 32, r, bounds, which, l, dy, "bf16", "f16", seed=7)
    gen = torch.Generator(device="cuda").manual_seed(m)
    xq = torch.randint(-3, 4, (m, k), generator=gen, device="cuda").to(torch.int8)
    xs = (2.0 ** torch.randint(-1, 2, (m, -(-k // 128)), generator=gen, device="cuda")).float()
    u = C.values((m, r), torch.float32, gen, True, 9)
    v = C.values((m, r), torch.float32, gen, True, 9)
    real = torch.zeros((m,), dtype=torch.bool, device="cuda")
    for rows, _ in C.owned(c):
        real[rows] = True
    u[~real], v[~real] = float("nan"), float("nan")  # never read
    c["dy"][~real] = float("nan")
    xhat = xq.double() * xs.double().repeat_interleave(128, 1)[:, :k]
    # units of 1/2: 9 . 3 . 2 a row, below 2^24 of them in all
    assert 2 * 9 * 3 * 2 * m < 2 ** 24
    return c, xq, xs, u, v, xhat


@pytest.mark.parametrize("dy", ["bf16", "f32"])
@pytest.mark.parametrize("name", SHAPES)
def test_whole_numbers(name, dy):
    c, xq, xs, u, v, xhat = make(name, dy)
    da64, db64 = C.grads64(c, xhat, u, v)
    args = (c["m"], c["k"], c["n"], c["l"], c["r"], c["dy"].dtype)
    size = w4.lora_grads_workspace_size(*args)
    whole = c["l"] * c["r"] * (c["k"] + c["n"]) * 4
    assert size >= 2 * whole and size % whole == 0  # two parts at least
    da, db = Canary(da64.shape, torch.float32), Canary(db64.shape, torch.float32)
    ws = Canary((size,), torch.uint8)
    da.tensor.fill_(5.0), db.tensor.fill_(5.0)
    p = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    status = _lib.load().lora_grads(p(xq), p(xs), c["m"], c["k"], p(c["dy"]), _lib._DT[c["dy"].dtype], c["n"], p(u), p(v),
                                    p(c["offsets"]), p(c["which"]), len(c["ids"]), c["l"], c["r"], p(da.tensor), p(db.tensor),
                                    p(ws.tensor), size, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert status == w4.W4_OK
    for t in (da, db, ws):
        t.check()
    assert torch.equal(da.tensor, da64.float()) and torch.equal(db.tensor, db64.float())
    # the wrapper gives the same
    got = w4.lora_grads(xq, xs, c["dy"], u, v, c["offsets"], c["which"], c["l"])
    assert torch.equal(got[0], da.tensor) and torch.equal(got[1], db.tensor)


@pytest.mark.parametrize("dy", ["bf16", "f32"])
def test_random(dy):
    c = C.case(2049, 322, 1056, 32, 40, [0, 700, 2049], [1, 0], 2, dy, "bf16", "f16", whole=False, seed=4)
    xq, xs = w4.quantize_checkpoint_int8(c["x"])
    gen = torch.Generator(device="cuda").manual_seed(5)
    u, v = C.values((2049, 40), torch.float32, gen, False), C.values((2049, 40), torch.float32, gen, False)
    xhat = xq.double() * xs.double().repeat_interleave(128, 1)[:, :1056]
    da64, db64 = C.grads64(c, xhat, u, v)
    da, db = w4.lora_grads(xq, xs, c["dy"], u, v, c["offsets"], c["which"], 2)
    assert w4.lora_grads_workspace_size(2049, 1056, 322, 2, 40, c["dy"].dtype) > 0
    assert C.rel(da, da64) <= C.sum_tol(2049) and C.rel(db, db64) <= C.sum_tol(2049)


def test_captured_and_replayed():
    """A captured call with its workspace, replayed with other requests in the same buffers; two graphs of one pool."""
    c, xq, xs, u, v, xhat = make("wide", "bf16")
    u, v = u.nan_to_num(0.0), v.nan_to_num(0.0)
    dy = c["dy"].nan_to_num(0.0)
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], None
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(w4.lora_grads(xq, xs, dy, u, v, c["offsets"], c["which"], 2))
        pool = g.pool()
        graphs.append(g)
    for bounds, which in (([0, 600, 1100], [1, 0]), ([7, 8, 1099], [0, -1]), ([0, 0, 1100], [1, 1]), ([0, 1100, 1100], [1, 0])):
        c["offsets"].copy_(torch.tensor(bounds, dtype=torch.int32))
        c["which"].copy_(torch.tensor(which, dtype=torch.int32))
        want = C.grads64({**c, "dy": dy, "bounds": bounds, "ids": which}, xhat, u, v)
        for g, out in zip(graphs, outs):
            for _ in range(2):
                g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0].float()) and torch.equal(out[1], want[1].float())
