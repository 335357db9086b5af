"""The way into the rank (u = scaling x A^T) in every tile of its kernels, bit for bit on whole numbers: the calls are chosen
so that the rule of w4a16_lora_matmul picks 16, 32 and 64 ranks a workgroup, for every pair of types, with K that ends
inside a wave's step, ranks that fill no tile, and ragged requests."""
import pytest
import torch

import dequant_gemm_quantize_amd as w4
from tests import lora_cases as C
from tests.gpu_util import Canary

pytestmark = pytest.mark.gpu


def tile(m, segments, rank):
    """The kernel that the rule picks: the least rounds of 256 workgroups times what a round reads; 4 rows and ranks a
    workgroup only where they save a fifth."""
    def cost(rows, ranks):
        tiles = (m + min(segments, m) * (rows - 1)) // rows * -(-rank // ranks)
        return -(-tiles // 256) * (rows + ranks)
    costs = [cost(16, 16), cost(16, 32), cost(16, 64)]
    if all(5 * cost(4, 4) <= 4 * c for c in costs):
        return 4
    if costs[0] <= costs[1] and costs[0] <= costs[2]:
        return 16
    return 32 if costs[1] <= costs[2] else 64


# rows, requests, rank, in, ranks a workgroup
CASES = [(2048, 9, 64, 1056, 64), (1700, 5, 72, 1056, 64), (1250, 5, 104, 2080, 64), (950, 5, 136, 544, 64), (800, 5, 256, 288, 64),
         (2750, 5, 40, 1312, 64), (2000, 5, 24, 1056, 32), (1400, 5, 40, 1312, 32), (1100, 5, 64, 544, 32), (800, 5, 72, 2080, 32),
         (200, 5, 256, 1056, 32), (1000, 2, 16, 1056, 16), (4500, 2, 16, 96, 16), (350, 5, 40, 32, 16), (300, 3, 16, 1056, 4)]


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")], ids="-".join)
@pytest.mark.parametrize("m,s,r,k,ranks", CASES)
def test_whole_numbers(m, s, r, k, ranks, types):
    assert tile(m, s, r) == ranks
    cuts = [m * i * i // (s * s) for i in range(s + 1)]  # ragged, the first request the shortest
    cuts[0], cuts[-1] = 2, m - 3
    c = C.case(m, 32, k, 32, r, cuts, [i % 4 - 1 if i else 2 for i in range(s)], 3, types[0], types[1], "f16", seed=r)
    y64, u64 = C.forward64(c)
    assert float(y64.abs().max()) < 2 ** 23
    y, u = Canary((m, 32), torch.float32), Canary((m, r), torch.float32)
    u.tensor.fill_(-77.0)
    w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"], out=y.tensor, u=u.tensor)
    y.check(), u.check()
    none = torch.ones((m,), dtype=torch.bool, device="cuda")
    for rows, _ in C.owned(c):
        none[rows] = False
        assert torch.equal(u.tensor[rows], u64[rows].float())
    assert (u.tensor[none] == -77.0).all() and torch.equal(y.tensor, y64.float())


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")], ids="-".join)
@pytest.mark.parametrize("m,s,r,k,ranks", CASES[:2] + CASES[7:8])
def test_random(m, s, r, k, ranks, types):
    c = C.case(m, 32, k, 32, r, [m * i // s for i in range(s + 1)], [i % 3 for i in range(s)], 3, types[0], types[1], "f16",
               whole=False, seed=k)
    u = torch.zeros((m, r), device="cuda")
    w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"], u=u)
    assert C.rel(u, C.forward64(c)[1]) <= C.sum_tol(k)
