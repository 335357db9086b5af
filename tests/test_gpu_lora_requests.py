"""Many requests of a row or a few in one call of many rows, forward: every row its own adapter, beside others of none, in
both tile sizes, with split sums and without, bit for bit on whole numbers."""
import pytest
import torch

import dequant_gemm_quantize_amd as w4
from tests import lora_cases as C
from tests.gpu_util import Canary

pytestmark = pytest.mark.gpu

# rows, out, in, group, rank, requests: above 64 rows and 2^31 products, up to 512 rows in tiles of 64 rows, then of 128
SHAPES = [(128, 2056, 8192, 128, 16, 128), (256, 4104, 2112, 64, 64, 256), (600, 2051, 2048, 128, 24, 600), (1100, 2050, 992, 32, 8, 500),
          (300, 2056, 4096, 128, 40, 77), (700, 4100, 768, 96, 16, 333)]


@pytest.mark.parametrize("ab", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k,g,r,s", SHAPES)
def test_whole_numbers(m, n, k, g, r, s, ab):
    gen = torch.Generator().manual_seed(s)
    cuts = torch.cat([torch.zeros(1, dtype=torch.int64), (torch.randperm(m - 1, generator=gen)[:s - 1] + 1).sort().values, torch.tensor([m])]).tolist()
    which = torch.randint(-1, 7, (s,), generator=gen).tolist()  # six adapters; -1 and 6 stand for none
    c = C.case(m, n, k, g, r, cuts, which, 6, "bf16", ab, "f16", seed=s)
    y64, u64 = C.forward64(c)
    assert float(y64.abs().max()) < 2 ** 23
    for dt in (torch.float32, torch.bfloat16):
        y, u = Canary((m, n), dt), torch.zeros((m, r), device="cuda")
        w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"], out=y.tensor, u=u)
        y.check()
        assert torch.equal(y.tensor, y64.to(dt)) and torch.equal(u, u64.float())


def test_adapters_that_are_not_numbers_stay_alone():
    """Every other request of a row has an adapter of NaN and infinities: the rows between keep their results."""
    m, n, k = 200, 2056, 5632
    c = C.case(m, n, k, 128, 16, list(range(m + 1)), [i % 2 for i in range(m)], 2)
    a, b, *rest = c["adapter"]
    a, b = a.clone(), b.clone()
    a[1, ::3], a[1, 1::3], b[1, ::2], b[1, 1::2] = float("nan"), float("inf"), float("nan"), float("-inf")
    y = w4.w4a16_lora_matmul(c["x"], *c["weight"], a, b, *rest)
    assert torch.equal(y[0::2], C.forward64(c)[0].bfloat16()[0::2])
    assert not y[1::2].isfinite().any()


def test_weights_beyond_4_gb():
    """[2^18 + 8, 2^15] codes, 4.3 GB, many rows: the last weight rows."""
    n, k, m = (1 << 18) + 8, 1 << 15, 70
    packed = torch.full((n, k // 2), 0x88, dtype=torch.uint8, device="cuda")  # weight 0 but for the last rows
    scales, zeros = torch.ones((n, k // 128), dtype=torch.float16, device="cuda"), torch.full((n, k // 128), 8.0, dtype=torch.float16, device="cuda")
    packed[-3:] = torch.randint(0, 256, (3, k // 2), device="cuda").to(torch.uint8)
    q = torch.stack([packed[-3:] & 15, packed[-3:] >> 4], -1).reshape(3, k).double() - 8
    x = torch.randint(-1, 2, (m, k), device="cuda").bfloat16()
    a = torch.randint(-1, 2, (2, 8, k), device="cuda").bfloat16()
    b = torch.zeros((2, n, 8), dtype=torch.bfloat16, device="cuda")
    b[1, -2:] = 1
    off, ad = torch.tensor([0, 69, m], dtype=torch.int32, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    y = w4.w4a16_lora_matmul(x, packed, scales, zeros, 128, a, b, torch.ones(2, device="cuda"), off, ad, out_dtype=torch.float32)
    want = x.double() @ q.t()
    want[-1, -2:] += (x[-1:].double() @ a[1].double().t()).sum()
    assert torch.equal(y[:, -3:], want.float()) and not y[:, :-3].any()
