"""The transposed products with any number of weight rows: rows of dy that do not start at 16-byte addresses, bit for bit
on whole numbers, in tiles of both sizes, with split sums and without, and where an odd number of fp16 scales leaves the
call to the kernel for few rows."""
import pytest
import torch

import dequant_gemm_quantize_amd as w4
from tests import lora_cases as C
from tests.gpu_util import Canary

pytestmark = pytest.mark.gpu

# rows, out, in, group: above 64 rows and 3 . 2^29 products in tiles; the last three by the kernel for few rows
SHAPES = [(100, 8001, 2112, 32), (129, 4097, 4096, 128), (300, 2051, 2816, 64), (1030, 2050, 1056, 96), (65, 8190, 4128, 32),
          (2100, 515, 2176, 128), (400, 1023, 4224, 4224), (9000, 33, 5632, 128), (70, 2051, 512, 128), (66, 2047, 96, 32),
          (257, 9, 32, 32)]


@pytest.mark.parametrize("types", [("bf16", "bf16", "f16"), ("bf16", "f32", "f32")], ids="-".join)
@pytest.mark.parametrize("m,n,k,g", SHAPES, ids=lambda v: str(v))
def test_whole_numbers(m, n, k, g, types):
    c = C.case(m, n, k, g, 24, [0, 5, 5, m // 3, m // 3 + 20, m - 3], [1, 0, -1, 2, 0], 3, *types, seed=m)
    dx64, v64 = C.back64(c)
    assert float(dx64.abs().max()) < 2 ** 23
    for dt in (torch.float32, torch.bfloat16):
        dx, v = Canary((m, k), dt), torch.zeros((m, 24), device="cuda")
        w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], *c["adapter"], out=dx.tensor, v=v)
        dx.check()
        assert torch.equal(dx.tensor, dx64.to(dt)) and torch.equal(v, v64.float())
        assert torch.equal(w4.w4a16_matmul_t(c["dy"], *c["weight"], out_dtype=dt), (c["dy"].double() @ c["dense"]).to(dt))


@pytest.mark.parametrize("m,n,k", [(300, 2051, 2816), (700, 1001, 2560)])
def test_captured_and_replayed(m, n, k):
    """The copy of dy is part of a captured call: replays with other dy in the same buffer, two graphs of one pool."""
    c = C.case(m, n, k, 128, 16, [0, m // 2, m], [1, 0], 2, seed=3)
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], None
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], *c["adapter"]))
        pool = g.pool()
        graphs.append(g)
    for turn in range(3):
        c["dy"].copy_(torch.randint(-1, 2, (m, n), device="cuda"))
        want = C.back64(c)[0].bfloat16()
        for g, out in zip(graphs, outs):
            for _ in range(2):
                g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), turn


def test_rows_that_are_not_numbers_stay_alone():
    m, n, k = 300, 2051, 2816
    c = C.case(m, n, k, 32, 16, [0, m // 2, m], [0, 1], 2)
    bad = m // 3
    dy = c["dy"].clone()
    dy[bad, ::3], dy[bad, 1::3] = float("nan"), float("-inf")
    dx = w4.w4a16_lora_matmul_t(dy, *c["weight"], *c["adapter"])
    keep = torch.arange(m, device="cuda") != bad
    assert torch.equal(dx[keep], C.back64(c)[0].bfloat16()[keep]) and dx[bad].isnan().any()


def test_rows_beyond_4_gb():
    """2^17 + 5 rows of 2^14 + 1 values, 4.3 GB of dy and of its copy: the last rows."""
    m, n, k = (1 << 17) + 5, (1 << 14) + 1, 64
    c = C.case(8, n, k, 32, 8, [0, 8], [1], 2)
    dy = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
    dy[-8:] = c["dy"]
    off = torch.tensor([0, m - 8, m], dtype=torch.int32, device="cuda")
    ad = torch.tensor([-1, 1], dtype=torch.int32, device="cuda")
    dx = w4.w4a16_lora_matmul_t(dy, *c["weight"], c["a"], c["b"], c["scaling"], off, ad, out_dtype=torch.float32)
    assert torch.equal(dx[-8:], C.back64(c)[0].float()) and not dx[:-8].any()
