"""Products with low-rank adapters, the transposed product and the adapters' gradients against their definition in 64
bits: bit for bit on whole numbers, within derived bounds on random ones."""
import pytest
import torch

import dequant_gemm_quantize_amd as w4
from tests import lora_cases as C
from tests.gpu_util import Canary

pytestmark = pytest.mark.gpu

# rows, out, in, group, rank, bounds, adapters of the segments, number of adapters
SHAPES = {
    "one row": (1, 32, 32, 32, 8, [0, 1], [0], 1),
    "one row of two adapters": (1, 256, 256, 128, 16, [0, 1], [1], 2),
    "three rows, one without": (3, 100, 64, 32, 8, [0, 1, 2, 3], [1, -1, 0], 2),
    "empty segments": (5, 33, 96, 32, 24, [0, 0, 2, 2, 2, 5, 5], [2, 0, 1, 1, 2, 0], 3),
    "rows before and behind": (40, 130, 160, 32, 8, [3, 10, 31], [1, 0], 2),
    "the same adapter twice": (50, 64, 256, 64, 16, [0, 7, 20, 50], [1, 0, 1], 2),
    "a number past the last adapter": (20, 48, 128, 128, 8, [0, 9, 20], [5, 1], 2),
    "widths that are odd": (37, 2051, 320, 64, 40, [0, 20, 37], [0, 1], 2),
    "many rows": (300, 520, 512, 128, 16, [0, 100, 300], [1, 0], 2),
    "many rows, units of 64": (129, 384, 576, 64, 32, [0, 128, 129], [0, 1], 2),
    "many rows, units of 32": (200, 200, 448, 32, 72, [5, 64, 190], [2, 0], 3),
    "segments of a row": (70, 96, 256, 128, 8, list(range(71)), [(7 * i) % 5 - 1 for i in range(70)], 4),
    "long columns": (9, 40, 2304, 96, 128, [0, 4, 9], [0, 1], 2),
    "no segments": (20, 64, 128, 64, 8, [0], [], 2),
    "groups as long as a row": (18, 70, 768, 768, 256, [0, 18], [0], 1),
}
TYPES = [("bf16", "bf16", "f16"), ("bf16", "f32", "f32"), ("f32", "f32", "f16"), ("f32", "bf16", "f32")]


def make(name, types, whole=True, seed=0):
    m, n, k, g, r, bounds, which, l = SHAPES[name]
    return C.case(m, n, k, g, r, bounds, which, l, *types, whole=whole, seed=seed)


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("name", SHAPES)
def test_whole_numbers_forward(name, types):
    c = make(name, types)
    y64, u64 = C.forward64(c)
    for dt in (torch.float32, torch.bfloat16):
        y, u = Canary((c["m"], c["n"]), dt), Canary((c["m"], c["r"]), torch.float32)
        u.tensor.fill_(-77.0)
        got = w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"], out=y.tensor, u=u.tensor)
        y.check(), u.check()
        assert torch.equal(got, y64.to(dt))
        none = torch.ones((c["m"],), dtype=torch.bool, device="cuda")
        for rows, _ in C.owned(c):
            none[rows] = False
            assert torch.equal(u.tensor[rows], u64[rows].float())
        assert (u.tensor[none] == -77.0).all()


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("name", SHAPES)
def test_whole_numbers_back(name, types):
    c = make(name, types)
    dx64, v64 = C.back64(c)
    plain64 = c["dy"].double() @ c["dense"]
    for dt in (torch.float32, torch.bfloat16):
        dx, v = Canary((c["m"], c["k"]), dt), Canary((c["m"], c["r"]), torch.float32)
        v.tensor.fill_(-77.0)
        w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], *c["adapter"], out=dx.tensor, v=v.tensor)
        dx.check(), v.check()
        assert torch.equal(dx.tensor, dx64.to(dt))
        for rows, _ in C.owned(c):
            assert torch.equal(v.tensor[rows], v64[rows].float())
        dx = Canary((c["m"], c["k"]), dt)
        w4.w4a16_matmul_t(c["dy"], *c["weight"], out=dx.tensor)
        dx.check()
        assert torch.equal(dx.tensor, plain64.to(dt))


@pytest.mark.parametrize("dy", ["bf16", "f32"])
@pytest.mark.parametrize("name", SHAPES)
def test_whole_numbers_grads(name, dy):
    c = make(name, (dy, "bf16", "f16"))
    gen = torch.Generator(device="cuda").manual_seed(3)
    nb = -(-c["k"] // 128)
    xq = torch.randint(-3, 4, (c["m"], c["k"]), generator=gen, device="cuda").to(torch.int8)
    xs = (2.0 ** torch.randint(-2, 3, (c["m"], nb), generator=gen, device="cuda")).float()
    u = C.values((c["m"], c["r"]), torch.float32, gen, True, 9)
    v = C.values((c["m"], c["r"]), torch.float32, gen, True, 9)
    real = torch.zeros((c["m"],), dtype=torch.bool, device="cuda")
    for rows, _ in C.owned(c):
        real[rows] = True
    u[~real], v[~real] = float("nan"), float("nan")  # never read
    dyn = c["dy"].clone()
    dyn[~real] = float("nan")
    xhat = xq.double() * xs.double().repeat_interleave(128, 1)[:, :c["k"]]
    da64, db64 = C.grads64(c, xhat, u, v)
    da, db = Canary(da64.shape, torch.float32), Canary(db64.shape, torch.float32)
    da.tensor.fill_(5.0), db.tensor.fill_(5.0)
    w4.lora_grads(xq, xs, dyn, u, v, c["offsets"], c["which"], c["l"], out=(da.tensor, db.tensor))
    da.check(), db.check()
    assert torch.equal(da.tensor, da64.float())
    assert torch.equal(db.tensor, db64.float())


def rounded(types):
    """Relative 2-norm bound of a bf16 result.  Its own rounding is at most half a step, 2^-8, of each element.  With bf16
    x the weights may be rounded too: a sum of terms t_i then misses the sum of t_i d_i, |d_i| <= 2^-8, independent
    and of mean zero, whose mean square is at most 2^-16 sum t_i^2; terms of random signs have sum t_i^2 for the mean
    square of the sum itself, so over many elements that is 2^-8 of the result's norm at most (and by the square root of 3 less, the errors being spread over their range)."""
    return (2 if types[0] == "bf16" else 1) * C.HALF[torch.bfloat16]


RANDOM = ["widths that are odd", "many rows, units of 32", "segments of a row", "long columns", "many rows"]


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("name", RANDOM)
def test_random_forward(name, types):
    c = make(name, types, whole=False, seed=1)
    y64, u64 = C.forward64(c)
    u = torch.zeros((c["m"], c["r"]), dtype=torch.float32, device="cuda")
    y = w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"], out_dtype=torch.float32, u=u)
    assert C.rel(u, u64) <= C.sum_tol(c["k"])
    # a group's code sums are up to 31 / 7.5 of their part that stays, the same again for the sums' own steps
    assert C.rel(y, y64) <= 4 * C.sum_tol(c["k"])
    yb = w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"], out_dtype=torch.bfloat16)
    assert C.rel(yb, y64) <= rounded(types) + 4 * C.sum_tol(c["k"])


@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("name", RANDOM)
def test_random_back(name, types):
    c = make(name, types, whole=False, seed=2)
    dx64, v64 = C.back64(c)
    v = torch.zeros((c["m"], c["r"]), dtype=torch.float32, device="cuda")
    dx = w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], *c["adapter"], out_dtype=torch.float32, v=v)
    assert C.rel(v, v64) <= C.sum_tol(c["n"])
    assert C.rel(dx, dx64) <= C.sum_tol(c["n"])
    dxb = w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], *c["adapter"], out_dtype=torch.bfloat16)
    assert C.rel(dxb, dx64) <= rounded(types) + C.sum_tol(c["n"])


@pytest.mark.parametrize("dy", ["bf16", "f32"])
@pytest.mark.parametrize("name", RANDOM)
def test_random_grads(name, dy):
    c = make(name, (dy, "bf16", "f16"), whole=False, seed=4)
    xq, xs = w4.quantize_checkpoint_int8(c["x"])
    gen = torch.Generator(device="cuda").manual_seed(5)
    u, v = C.values((c["m"], c["r"]), torch.float32, gen, False), C.values((c["m"], c["r"]), torch.float32, gen, False)
    xhat = xq.double() * xs.double().repeat_interleave(128, 1)[:, :c["k"]]
    da64, db64 = C.grads64(c, xhat, u, v)
    da, db = w4.lora_grads(xq, xs, c["dy"], u, v, c["offsets"], c["which"], c["l"])
    assert C.rel(da, da64) <= C.sum_tol(c["m"]) and C.rel(db, db64) <= C.sum_tol(c["m"])


def test_a_training_run_of_the_operators():
    """Forward, checkpoint, gradient with respect to x and to the adapters, one after the other, as a step makes them."""
    c = make("many rows", ("bf16", "bf16", "f16"))
    y64, u64 = C.forward64(c)
    dx64, v64 = C.back64(c)
    u = torch.empty((c["m"], c["r"]), device="cuda")
    v = torch.empty_like(u)
    y = w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"], u=u)
    xq, xs = w4.quantize_checkpoint_int8(c["x"])
    dx = w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], *c["adapter"], v=v)
    da, db = w4.lora_grads(xq, xs, c["dy"], u, v, c["offsets"], c["which"], c["l"])
    assert torch.equal(y, y64.bfloat16()) and torch.equal(dx, dx64.bfloat16())
    xhat = w4.dequant_checkpoint_int8(xq, xs, out_dtype=torch.float32).double()
    da64, db64 = C.grads64(c, xhat, u64, v64)
    assert torch.equal(db, db64.float())
    assert C.rel(da, da64) <= C.sum_tol(c["m"])


# rows, out, in, group, x, adapters and scales: what the tiles take (forward above 64 rows and 2^31 products, back
# above 32 rows), by the edges of a tile (256 or 128 rows, 128 columns), of a step (64) and of the parts of a split sum
TILES = [
    (300, 2056, 4096, 128, ("bf16", "bf16", "f16")),   # split forward and back, ragged columns
    (300, 2051, 4096, 128, ("bf16", "bf16", "f16")),   # odd columns forward; back on the kernel for few rows
    (257, 11016, 1056, 96, ("bf16", "f32", "f32")),    # one part forward, groups across steps and tiles, K ends inside a step
    (129, 8200, 2080, 32, ("bf16", "bf16", "f16")),    # groups of 32, K ends inside a step
    (66, 10248, 3264, 64, ("bf16", "f32", "f16")),     # tiles of 128 rows, most of them empty
    (1025, 1032, 2112, 2112, ("bf16", "bf16", "f32")),  # groups as long as a row
    (700, 4104, 1024, 256, ("bf16", "bf16", "f16")),
    (40, 8, 32, 32, ("bf16", "bf16", "f16")),          # back: one step of eight rows
    (33, 72, 160, 32, ("bf16", "bf16", "f32")),
    (200, 4096, 32, 32, ("bf16", "f32", "f16")),       # back: a tile wider than the result
]


@pytest.mark.parametrize("m,n,k,g,types", TILES, ids=[f"{t[0]}x{t[1]}x{t[2]}g{t[3]}" for t in TILES])
def test_whole_numbers_in_tiles(m, n, k, g, types):
    bounds, which = [0, 5, 5, m // 3, m // 3 + 40 if m > 60 else m // 3 + 1, m - 3], [1, 0, -1, 2, 0]
    c = C.case(m, n, k, g, 24, bounds, which, 3, *types)
    y64, u64 = C.forward64(c)
    dx64, v64 = C.back64(c)
    assert float(y64.abs().max()) < 2 ** 23 and float(dx64.abs().max()) < 2 ** 23  # halves: 2^24 units
    for dt in (torch.float32, torch.bfloat16):
        y, dx = Canary((m, n), dt), Canary((m, k), dt)
        w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"], out=y.tensor)
        w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], *c["adapter"], out=dx.tensor)
        y.check(), dx.check()
        assert torch.equal(y.tensor, y64.to(dt))
        assert torch.equal(dx.tensor, dx64.to(dt))
        assert torch.equal(w4.w4a16_matmul_t(c["dy"], *c["weight"], out_dtype=dt), (c["dy"].double() @ c["dense"]).to(dt))


@pytest.mark.parametrize("m,n,k,g,types", TILES[:6], ids=[f"{t[0]}x{t[1]}x{t[2]}g{t[3]}" for t in TILES[:6]])
def test_random_in_tiles(m, n, k, g, types):
    c = C.case(m, n, k, g, 40, [0, m // 2, m], [1, 0], 2, *types, whole=False, seed=9)
    y64, _ = C.forward64(c)
    dx64, _ = C.back64(c)
    for dt, steps in ((torch.float32, 0.0), (torch.bfloat16, rounded(types))):
        y = w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"], out_dtype=dt)
        dx = w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], *c["adapter"], out_dtype=dt)
        assert C.rel(y, y64) <= steps + 4 * C.sum_tol(k)
        assert C.rel(dx, dx64) <= steps + C.sum_tol(n)


def test_rows_that_are_not_numbers_stay_alone():
    """A row with NaN and infinities beside others, in every kernel: the others' results do not change."""
    for m, n, k in ((300, 2056, 4096), (24, 264, 256), (3, 64, 96)):
        c = C.case(m, n, k, 32, 16, [0, m // 2, m], [0, 1], 2)
        bad = m // 3
        keep = torch.arange(m, device="cuda") != bad
        x, dy = c["x"].clone(), c["dy"].clone()
        x[bad, ::3], x[bad, 1::3] = float("nan"), float("inf")
        dy[bad, ::3], dy[bad, 1::3] = float("nan"), float("-inf")
        y = w4.w4a16_lora_matmul(x, *c["weight"], *c["adapter"])
        dx = w4.w4a16_lora_matmul_t(dy, *c["weight"], *c["adapter"])
        assert torch.equal(y[keep], C.forward64(c)[0].bfloat16()[keep])
        assert torch.equal(dx[keep], C.back64(c)[0].bfloat16()[keep])
        assert y[bad].isnan().any() and dx[bad].isnan().any()


def test_adapters_that_are_not_numbers_stay_alone():
    """One request's adapter holds NaN and infinities: the rows of the others do not change, in any kernel."""
    for m, n, k in ((300, 2056, 4096), (90, 2056, 512), (24, 264, 256), (3, 64, 96)):
        for ab in ("bf16", "f32"):
            c = C.case(m, n, k, 32, 24, [0, m // 3, 2 * m // 3, m], [0, 1, 2], 3, ab=ab)
            a, b, *rest = c["adapter"]
            a, b = a.clone(), b.clone()
            a[1, ::3], a[1, 1::3], b[1, ::2], b[1, 1::2] = float("nan"), float("inf"), float("nan"), float("-inf")
            keep = torch.ones(m, dtype=torch.bool, device="cuda")
            keep[m // 3:2 * m // 3] = False
            u, v = torch.zeros((m, 24), device="cuda"), torch.zeros((m, 24), device="cuda")
            y = w4.w4a16_lora_matmul(c["x"], *c["weight"], a, b, *rest, u=u)
            dx = w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], a, b, *rest, v=v)
            xq, xs = w4.quantize_checkpoint_int8(c["x"])
            da, db = w4.lora_grads(xq, xs, c["dy"], u, v, c["offsets"], c["which"], 3)
            assert torch.equal(y[keep], C.forward64(c)[0].bfloat16()[keep])
            assert torch.equal(dx[keep], C.back64(c)[0].bfloat16()[keep])
            assert not y[~keep].isfinite().any() and not dx[~keep].isfinite().any()
            assert da[0::2].isfinite().all() and db[0::2].isfinite().all()


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 9])
def test_segments_of_few_rows(rows):
    """Every number of rows that the vector kernel of the way into the rank has, more than 64 segments, twice the same adapter."""
    s = 70
    c = C.case(rows * s, 48, 1056, 96, 16, [rows * i for i in range(s + 1)], [i % 5 - 1 for i in range(s)], 4)
    u = torch.zeros((rows * s, 16), device="cuda")
    y64, u64 = C.forward64(c)
    y = w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"], out_dtype=torch.float32, u=u)
    assert torch.equal(u, u64.float()) and torch.equal(y, y64.float())
    v = torch.zeros_like(u)
    dx64, v64 = C.back64(c)
    dx = w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], *c["adapter"], out_dtype=torch.float32, v=v)
    assert torch.equal(v, v64.float()) and torch.equal(dx, dx64.float())


@pytest.mark.parametrize("m", [0, 4])
def test_empty_calls(m):
    c = C.case(m, 32, 64, 32, 8, [0, m], [0], 1)
    assert w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"]).shape == (m, 32)
    assert w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], *c["adapter"]).shape == (m, 64)
    assert w4.w4a16_matmul_t(c["dy"], *c["weight"]).shape == (m, 64)
    xq, xs = w4.quantize_checkpoint_int8(c["x"])
    u = torch.zeros((m, 8), device="cuda")
    da, db = w4.lora_grads(xq, xs, c["dy"], u, u, c["offsets"], c["which"], 1)
    assert not da.any() and not db.any() and da.shape == (1, 8, 64) and db.shape == (1, 32, 8)
    none = w4.lora_grads(xq, xs, c["dy"], u, u, c["offsets"], c["which"], 0)
    assert none[0].shape == (0, 8, 64) and none[1].shape == (0, 32, 8)


def test_offsets_out_of_order_stay_in_bounds():
    """Every number that offsets and adapters may hold leads to memory of the call's own: results of such rows are
    unspecified, what lies around the outputs stays."""
    c = C.case(90, 70, 256, 128, 16, [0, 90], [0], 2)
    for bounds, which in [([50, 3, 90, -7], [0, 1, 0]), ([0, 2 ** 31 - 1, 10, 20], [1, 2 ** 31 - 1, -2 ** 31]),
                          ([-2 ** 31, -5, 200, 91], [0, 0, 1]), ([90, 90, 90, 0], [1, 1, 1])]:
        ad = (c["a"], c["b"], c["scaling"], torch.tensor(bounds, dtype=torch.int32, device="cuda"),
              torch.tensor(which, dtype=torch.int32, device="cuda"))
        for x, dy in ((c["x"], c["dy"]), (c["x"][:9], c["dy"][:9])):
            m = x.shape[0]
            y, u = Canary((m, 70), torch.bfloat16), Canary((m, 16), torch.float32)
            dx, v = Canary((m, 256), torch.bfloat16), Canary((m, 16), torch.float32)
            da, db = Canary((2, 16, 256), torch.float32), Canary((2, 70, 16), torch.float32)
            w4.w4a16_lora_matmul(x, *c["weight"], *ad, out=y.tensor, u=u.tensor)
            w4.w4a16_lora_matmul_t(dy, *c["weight"], *ad, out=dx.tensor, v=v.tensor)
            xq, xs = w4.quantize_checkpoint_int8(x)
            w4.lora_grads(xq, xs, dy, u.tensor, v.tensor, *ad[3:], 2, out=(da.tensor, db.tensor))
            for t in (y, u, dx, v, da, db):
                t.check()
