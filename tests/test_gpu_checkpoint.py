"""quantize_checkpoint_int8 and dequant_checkpoint_int8 against their definition in 64 bits."""
import numpy as np
import pytest
import torch

import dequant_gemm_quantize_amd as w4
from tests.gpu_util import Canary

pytestmark = pytest.mark.gpu
B = 128


def definition(x):
    """Codes and scales of float32 / bf16 rows on the CPU: the scale one float32 division, the code from the exact
    quotient.  A float64 quotient of a float32 by a float32 is a half-integer only if the exact one is: otherwise
    x differs from (c + 1/2) s by a unit of x or s at least, 2^-32 of the quotient or more."""
    x = x.float().cpu().numpy().astype(np.float32)
    m, k = x.shape
    nb = -(-k // B)
    pad = np.zeros((m, nb * B), np.float32)
    pad[:, :k] = x
    blk = pad.reshape(m, nb, B)
    with np.errstate(all="ignore"):
        s = np.abs(blk).max(-1) / np.float32(127)
        bad = ~np.isfinite(blk).all(-1)
        s[bad] = np.nan
        q = np.where((s > 0)[..., None], np.rint(blk.astype(np.float64) / s.astype(np.float64)[..., None]), 0)
    q = np.where(bad[..., None], 0, np.clip(q, -127, 127))
    return q.reshape(m, -1)[:, :k].astype(np.int8), s.astype(np.float32)


def check(x):
    xq, xs = w4.quantize_checkpoint_int8(x)
    q, s = definition(x)
    assert np.array_equal(xs.cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(xq.cpu().numpy(), q)
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        got = w4.dequant_checkpoint_int8(xq, xs, out_dtype=dt)
        want = (xq.cpu().float() * torch.from_numpy(s).repeat_interleave(B, 1)[:, :x.shape[1]]).to(dt)
        assert torch.equal(got.cpu().nan_to_num(7.0), want.nan_to_num(7.0))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,k", [(1, 32), (3, 96), (1, 128), (5, 160), (17, 512), (2, 4096), (33, 11008), (257, 224)])
def test_random_rows(m, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(m * k)
    x = torch.randn((m, k), generator=gen, device="cuda") * torch.exp2(torch.randint(-20, 20, (m, 1), generator=gen,
                                                                                    device="cuda").float())
    x = torch.where(torch.rand((k,), generator=gen, device="cuda") < 0.05, x * 20, x)
    check(x.to(dtype))


def test_borders():
    """Quotients on, just above and just below every half-integer, at scales that are no powers of two."""
    rows = []
    for top in (127.0, 1.0, 3.1415927, 1e-3, 5e7):
        s = np.float32(np.float32(top) / np.float32(127))
        mid = ((np.arange(126) + 0.5) * np.float64(s)).astype(np.float32)
        for step in (-1, 0, 1):
            v = mid if step == 0 else np.nextafter(mid, np.float32(np.inf if step > 0 else -np.inf))
            rows.append(np.concatenate([v, [top, 0]]).astype(np.float32))
            rows.append(-rows[-1])
    check(torch.from_numpy(np.stack(rows)).cuda())


def test_extremes():
    """Zeros, subnormal blocks, the largest values, negative zeros."""
    x = np.zeros((9, 256), np.float32)
    x[1, 5] = -0.0
    x[2, :128] = np.float32(1e-45) * np.arange(128)  # scales of zero or one smallest step
    x[3, :128] = np.float32(1e-45) * np.arange(60)[:, None].repeat(3, 1).reshape(-1)[:128]
    x[4, :] = np.finfo(np.float32).max
    x[5, ::2] = -np.finfo(np.float32).max
    x[6, :] = np.float32(2.0 ** -126)
    x[7, :128] = np.float32(2.0 ** -60) * np.linspace(-1, 1, 128, dtype=np.float32)
    x[8, 128:] = np.float32(2.0 ** -66) * np.linspace(-1, 1, 128, dtype=np.float32)
    check(torch.from_numpy(x).cuda())


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_not_numbers_stay_in_their_block(bad):
    x = torch.randn((3, 288), device="cuda")
    x[1, 130] = bad
    check(x)
    xq, xs = w4.quantize_checkpoint_int8(x)
    v = w4.dequant_checkpoint_int8(xq, xs, out_dtype=torch.float32)
    assert v[1, 128:256].isnan().all() and not v[1, :128].isnan().any() and not v[1, 256:].isnan().any()


def test_empty_and_outputs():
    x = torch.zeros((0, 64), device="cuda")
    xq, xs = w4.quantize_checkpoint_int8(x)
    assert xq.shape == (0, 64) and xs.shape == (0, 1)
    assert w4.dequant_checkpoint_int8(xq, xs).shape == (0, 64)
    x = torch.randn((7, 160), device="cuda")
    cq, cs, cv = Canary((7, 160), torch.int8), Canary((7, 2), torch.float32), Canary((7, 160), torch.bfloat16)
    w4.quantize_checkpoint_int8(x, out=(cq.tensor, cs.tensor))
    w4.dequant_checkpoint_int8(cq.tensor, cs.tensor, out=cv.tensor)
    for c in (cq, cs, cv):
        c.check()
    assert torch.equal(cq.tensor, w4.quantize_checkpoint_int8(x)[0])


def test_more_blocks_than_a_launch_has_groups():
    """2^24 rows of 32 columns: every row is a block, 16 to a workgroup, 2^20 workgroups at a time."""
    m = 1 << 24
    x = torch.zeros((m, 32), dtype=torch.bfloat16, device="cuda")
    x[-1] = 3
    x[m // 2] = -2
    xq, xs = w4.quantize_checkpoint_int8(x)
    assert int(xq[-1].min()) == 127 and int(xq[m // 2].max()) == -127 and int((xq != 0).sum()) == 64
    assert float(xs[-1]) == float(torch.tensor(3.0) / 127)
    assert torch.equal(w4.dequant_checkpoint_int8(xq, xs), x)
