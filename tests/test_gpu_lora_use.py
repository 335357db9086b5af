"""Adapters as they are used: the layer and its gradients, streams, captured calls, more than 4 GB of an operand."""
import pytest
import torch

import dequant_gemm_quantize_amd as w4
from tests import lora_cases as C

pytestmark = pytest.mark.gpu


def layer(n=96, k=256, g=64, adapters=3, rank=8, dtype=torch.float32, seed=0):
    torch.manual_seed(seed)
    base = w4.QuantizedLinear.from_weight(torch.randn(n, k, device="cuda") * 0.05, group_size=g)
    lora = w4.LoRALinear(base, rank=rank, alpha=12.0, adapters=adapters, dtype=dtype)
    with torch.no_grad():
        lora.b.copy_(torch.randn_like(lora.b) * 0.1)
    return base, lora


def codes(m, k, dtype=torch.float32):
    """Activations that their 8-bit checkpoint holds exactly: whole numbers, 127 the largest of each block of 128."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randint(-126, 127, (m, k), generator=gen, device="cuda").to(dtype)
    x[:, ::128] = 127
    return x


def test_layer_against_dense_layers():
    base, lora = layer()
    x = codes(11, 256)
    offsets, which = torch.tensor([0, 3, 8, 11], dtype=torch.int32, device="cuda"), torch.tensor([2, -1, 0], dtype=torch.int32, device="cuda")
    y = lora(x.view(11, 1, 256), offsets, which)
    assert y.shape == (11, 1, 96) and y.dtype == torch.float32
    dense = base.dequantize(torch.float32).double()
    want = x.double() @ dense.t()
    for rows, l in ((slice(0, 3), 2), (slice(8, 11), 0)):
        want[rows] += 1.5 * (x[rows].double() @ lora.a[l].double().t()) @ lora.b[l].double().t()
    assert C.rel(y.view(11, 96), want) <= 4 * C.sum_tol(256)
    # one adapter for all rows
    y0 = lora(x)
    want = x.double() @ dense.t() + 1.5 * (x.double() @ lora.a[0].double().t()) @ lora.b[0].double().t()
    assert C.rel(y0, want) <= 4 * C.sum_tol(256)


def test_fresh_adapter_adds_nothing():
    base = w4.QuantizedLinear.from_weight(torch.randn(64, 128, device="cuda"), group_size=32)
    lora = w4.LoRALinear(base, rank=16)
    x = torch.randn(5, 128, device="cuda")
    assert C.rel(lora(x), base(x).double()) <= 4 * C.sum_tol(128)
    assert lora.packed.data_ptr() == base.packed.data_ptr()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_gradients_against_the_formula(dtype):
    base, lora = layer()
    x = codes(40, 256, dtype).requires_grad_()
    offsets, which = torch.tensor([0, 10, 25, 36], dtype=torch.int32, device="cuda"), torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    y = lora(x, offsets, which)
    assert y.dtype == dtype
    dy = torch.randn(40, 96, device="cuda").to(dtype)
    dx, da, db = torch.autograd.grad(y, (x, lora.a, lora.b), dy)
    dense = base.dequantize(torch.float32).double()
    d, a, b = dy.double(), lora.a.double(), lora.b.double()
    want_x, want_a, want_b = d @ dense, torch.zeros_like(a), torch.zeros_like(b)
    for rows, l in ((slice(0, 10), 1), (slice(10, 25), 0), (slice(25, 36), 1)):
        v, u = 1.5 * d[rows] @ b[l], 1.5 * x[rows].double() @ a[l].t()
        want_x[rows] += v @ a[l]
        want_a[l] += v.t().contiguous() @ x[rows].double()
        want_b[l] += d[rows].t().contiguous() @ u
    half = C.HALF[dtype]
    assert dx.dtype == dtype and C.rel(dx, want_x) <= (2 if dtype == torch.bfloat16 else 1) * half + 4 * C.sum_tol(96)
    assert C.rel(da, want_a) <= 4 * C.sum_tol(96) and C.rel(db, want_b) <= 4 * C.sum_tol(256)
    assert not da[2].any() and not db[2].any()  # an adapter without rows


def test_gradients_against_differences():
    """The loss is linear in each of x, a and b: a difference quotient is its derivative but for the float32 rounding of
    the two losses, 2^-24 sqrt(n) of sums of n terms each (sum_tol), relative to the loss's size over the step's."""
    _, lora = layer(seed=3)
    x = codes(30, 256).requires_grad_()
    dy = torch.randn(30, 96, device="cuda")
    grads = torch.autograd.grad(lora(x), (x, lora.a, lora.b), dy)
    for leaf, grad in zip((x, lora.a, lora.b), grads):
        step = torch.randn_like(leaf)
        if leaf is x:
            step = torch.randint(-3, 4, leaf.shape, device="cuda").float()
        elif leaf.shape[0] > 1:
            step[1:] = 0  # the rows have adapter 0
        with torch.no_grad():
            kept = leaf.detach().clone()
            losses = []
            for sign in (1, -1):
                leaf.copy_(kept + sign * step)
                losses.append((lora(x).double() * dy.double()).sum())
            leaf.copy_(kept)
            size = (lora(x).double() * dy.double()).abs().sum() + sum(abs(v) for v in losses)
        slope = (losses[0] - losses[1]) / 2
        want = (grad.double() * step.double()).sum()
        assert float((slope - want).abs()) <= 4 * C.sum_tol(256) * float(size) + 1e-6 * float(want.abs())


def test_nothing_is_kept_without_gradients():
    _, lora = layer()
    x = codes(6, 256)
    with torch.no_grad():
        assert lora(x).grad_fn is None
    lora.requires_grad_(False)
    assert lora(x).grad_fn is None
    saved = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: saved.append(t.dtype) or t, lambda t: t):
        y = lora(x.requires_grad_())
    assert torch.int8 not in saved  # x alone: no checkpoint among what is kept
    dx, = torch.autograd.grad(y, x, torch.ones_like(y))
    assert dx.shape == x.shape


def test_no_second_derivative():
    _, lora = layer()
    x = codes(6, 256).requires_grad_()
    dx, = torch.autograd.grad(lora(x).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


def test_training_step_runs_and_moves_the_adapters_alone():
    base, lora = layer(dtype=torch.bfloat16)
    before = [t.clone() for t in (lora.packed, lora.scales, lora.zeros)]
    opt = torch.optim.SGD(lora.parameters(), lr=0.1)
    a0, b0 = lora.a.detach().clone(), lora.b.detach().clone()
    x = torch.randn(4, 9, 256, device="cuda", dtype=torch.bfloat16)
    lora(x).float().pow(2).mean().backward()
    opt.step()
    assert not torch.equal(lora.a, a0) and not torch.equal(lora.b, b0)
    assert torch.equal(lora.a[1:], a0[1:])  # adapters without rows
    assert all(torch.equal(s, t) for s, t in zip(before, (lora.packed, lora.scales, lora.zeros)))


def test_layer_refusals():
    base = w4.QuantizedLinear.from_weight(torch.randn(64, 128, device="cuda"), group_size=32)
    for kw in ({"rank": 4}, {"rank": 264}, {"adapters": 0}, {"dtype": torch.float16}):
        with pytest.raises(ValueError):
            w4.LoRALinear(base, **kw)
    base.act_int8 = True
    with pytest.raises(ValueError):
        w4.LoRALinear(base)
    base.act_int8 = False
    lora = w4.LoRALinear(base)
    with pytest.raises(ValueError):
        lora(torch.randn(3, 96, device="cuda"))
    with pytest.raises(ValueError):
        lora(torch.randn(3, 128, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda"))


def run_all(c, u, v):
    y = w4.w4a16_lora_matmul(c["x"], *c["weight"], *c["adapter"], u=u)
    dx = w4.w4a16_lora_matmul_t(c["dy"], *c["weight"], *c["adapter"], v=v)
    xq, xs = w4.quantize_checkpoint_int8(c["x"])
    return (y, dx, *w4.lora_grads(xq, xs, c["dy"], u, v, c["offsets"], c["which"], c["l"]))


@pytest.mark.parametrize("m,n,k", [(9, 264, 512), (200, 4104, 4096)])
def test_side_stream(m, n, k):
    """Tensors made on the default stream, used on another, two calls at once on two streams."""
    c = C.case(m, n, k, 128, 16, [0, m // 2, m], [1, 0], 2)
    low = [torch.zeros((m, 16), device="cuda") for _ in range(4)]
    want = run_all(c, low[0], low[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got.append(run_all(c, low[2 * i], low[2 * i + 1]))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(p, q) for p, q in zip(g, want))


@pytest.mark.parametrize("m,n,k", [(9, 264, 512), (200, 4104, 4096)])
def test_captured_and_replayed(m, n, k):
    """A captured step (first calls of their kind, split sums with workspaces) replayed with other segments, adapters and
    activations in the same buffers, with eager work between; two graphs of one memory pool."""
    c = C.case(m, n, k, 64, 32, [0, m // 2, m], [1, 0], 3, seed=5)
    u, v = torch.zeros((m, 32), device="cuda"), torch.zeros((m, 32), device="cuda")
    torch.cuda.synchronize()
    graphs, outs = [], []
    pool = None
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(run_all(c, u, v))
        pool = g.pool()
        graphs.append(g)
    for turn, (bounds, which) in enumerate([([0, m // 2, m], [1, 0]), ([0, 1, m], [2, 2]), ([2, 5, m - 1], [0, -1]), ([0, 0, m], [0, 1])]):
        c["offsets"].copy_(torch.tensor(bounds, dtype=torch.int32))
        c["which"].copy_(torch.tensor(which, dtype=torch.int32))
        c["x"].copy_(torch.randint(-1, 2, (m, k), device="cuda"))
        eager = run_all(c, torch.zeros_like(u), torch.zeros_like(v))
        for g, out in zip(graphs, outs):
            for _ in range(2):
                g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(out, eager)), turn


def test_captured_training_step():
    """Forward and backward of the layer in one graph, warmed up on the capturing stream, replayed against eager."""
    _, lora = layer(n=264, k=512)
    x = codes(50, 512)
    dy = torch.randn(50, 264, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.autograd.grad(lora(x), (lora.a, lora.b), dy)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lora(x)
        da, db = torch.autograd.grad(y, (lora.a, lora.b), dy)
    for _ in range(3):
        dy.copy_(torch.randn_like(dy))
        g.replay()
        torch.cuda.synchronize()
        ye = lora(x)
        dae, dbe = torch.autograd.grad(ye, (lora.a, lora.b), dy)
        assert torch.equal(y, ye) and torch.equal(da, dae) and torch.equal(db, dbe)


def test_same_result_every_time():
    c = C.case(333, 2056, 2112, 64, 40, [0, 100, 333], [1, 0], 2, whole=False, seed=11)
    u, v = torch.zeros((333, 40), device="cuda"), torch.zeros((333, 40), device="cuda")
    first = [t.clone() for t in run_all(c, u, v)]
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(first, run_all(c, u, v)))


def test_weights_and_adapters_beyond_4_gb():
    """[2^18 + 8, 2^15] codes, 4.3 GB, and 300 adapters of rank 256, 5 GB: the last rows of both."""
    n, k, m, l, r = (1 << 18) + 8, 1 << 15, 40, 300, 256
    packed = torch.full((n, k // 2), 0x88, dtype=torch.uint8, device="cuda")  # weight 0 ...
    scales, zeros = torch.ones((n, k // 128), dtype=torch.float16, device="cuda"), torch.full((n, k // 128), 8.0, dtype=torch.float16, device="cuda")
    packed[-3:] = torch.randint(0, 256, (3, k // 2), device="cuda").to(torch.uint8)  # ... but for the last rows
    q = torch.stack([packed[-3:] & 15, packed[-3:] >> 4], -1).reshape(3, k).double() - 8
    dy = torch.randint(-2, 3, (m, n), device="cuda").bfloat16()
    want = dy[:, -3:].double() @ q
    assert torch.equal(w4.w4a16_matmul_t(dy, packed, scales, zeros, 128, out_dtype=torch.float32), want.float())
    assert torch.equal(w4.w4a16_matmul_t(dy[:4], packed, scales, zeros, 128, out_dtype=torch.float32), want[:4].float())
    x = torch.randint(-1, 2, (m, k), device="cuda").bfloat16()
    a = torch.zeros((l, r, k), dtype=torch.bfloat16, device="cuda")
    a[-1] = torch.randint(-1, 2, (r, k), device="cuda").bfloat16()
    b = torch.ones((l, 64, r), dtype=torch.bfloat16, device="cuda")
    off, ad = torch.tensor([0, m], dtype=torch.int32, device="cuda"), torch.tensor([l - 1], dtype=torch.int32, device="cuda")
    args = (packed[-64:].contiguous(), scales[-64:].contiguous(), zeros[-64:].contiguous(), 128, a, b,
            torch.ones(l, device="cuda"), off, ad)
    y = w4.w4a16_lora_matmul(x, *args, out_dtype=torch.float32)
    want = (x.double() @ a[-1].double().t()).sum(1, keepdim=True).expand(m, 64).clone()
    want[:, -3:] += x.double() @ q.t()
    assert torch.equal(y, want.float())
    d = torch.randint(-1, 2, (m, 64), device="cuda").bfloat16()
    dx = w4.w4a16_lora_matmul_t(d, *args, out_dtype=torch.float32)
    want = d.double().sum(1, keepdim=True) * a[-1].double().sum(0) + d[:, -3:].double() @ q
    assert torch.equal(dx, want.float())


def test_rows_beyond_4_gb():
    """2^17 + 5 rows of 2^15 columns, 8.6 GB of x: the last rows."""
    m, k, n = (1 << 17) + 5, 1 << 15, 32
    c = C.case(8, n, k, 128, 8, [0, 8], [1], 2)
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    x[-8:] = c["x"]
    off = torch.tensor([0, m - 8, m], dtype=torch.int32, device="cuda")
    ad = torch.tensor([-1, 1], dtype=torch.int32, device="cuda")
    u = torch.zeros((m, 8), device="cuda")
    y = w4.w4a16_lora_matmul(x, *c["weight"], c["a"], c["b"], c["scaling"], off, ad, out_dtype=torch.float32, u=u)
    y64, u64 = C.forward64(c)
    assert torch.equal(y[-8:], y64.float()) and torch.equal(u[-8:], u64.float()) and not y[:-8].any()
    xq, xs = w4.quantize_checkpoint_int8(x)
    assert torch.equal(w4.dequant_checkpoint_int8(xq[-8:].contiguous(), xs[-8:].contiguous(), out_dtype=torch.float32), c["x"].float())
    dy = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
    dy[-8:] = c["dy"]
    v = torch.zeros((m, 8), device="cuda")
    v[-8:] = 1.0
    da, db = w4.lora_grads(xq, xs, dy, u, v, off, ad, 2)
    da64, db64 = C.grads64(c, c["x"].double(), u64, v[-8:])
    assert torch.equal(da, da64.float()) and torch.equal(db, db64.float())
