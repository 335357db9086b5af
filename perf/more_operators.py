"""Cases of training and serving low-rank adapters beside a frozen INT4 weight, each in a plain form and as the library's calls.

Operators:
  lora         w4a16_lora_matmul: the INT4 projection and, on top, the adapter of each request, requests mixed in one batch
  back         w4a16_matmul_t and w4a16_lora_matmul_t: the gradient with respect to x through the frozen weight (and the adapters)
  checkpoint   quantize_checkpoint_int8 then dequant_checkpoint_int8: the values that the 8-bit codes and block scales stand for
  grads        lora_grads: the adapters' gradients from the 8-bit checkpoint of x
  step         lora_linear: a layer's forward and backward, which makes all of these calls
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128  # columns of a block of the 8-bit checkpoint
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    lora = {"op": "lora", "g": 128, "sz": "f16", "x": "bf16", "ab": "bf16", "out": "bf16", "none": 0.0, "behind": 0}
    back = {**lora, "op": "back"}
    grads = {"op": "grads", "x": "bf16", "dy": "bf16", "none": 0.0, "behind": 0}
    return [
        # decode of one request with its adapter, Llama-7B up projection
        {**lora, "name": "lora 1 token", "m": 1, "n": 11008, "k": 4096, "r": 16, "l": 8, "s": 1},
        # decode of 64 requests, one token each, 32 adapters (some requests without one), down projection
        {**lora, "name": "lora 64 requests", "m": 64, "n": 4096, "k": 11008, "r": 16, "l": 32, "s": 64, "none": 0.2},
        # a small fp32 layer with odd widths, groups of 64 and a padded batch
        {**lora, "name": "lora 77 rows f32", "m": 77, "n": 2050, "k": 2048, "g": 64, "r": 8, "l": 4, "s": 5, "x": "f32",
         "ab": "f32", "out": "f32", "sz": "f32", "none": 0.2, "behind": 9},
        # prefill of nine requests, up projection
        {**lora, "name": "lora 2048 rows", "m": 2048, "n": 11008, "k": 4096, "r": 64, "l": 8, "s": 9},
        # the gradient of a few rows (a reward on the last tokens), adapters included
        {**back, "name": "back 12 rows", "m": 12, "n": 11008, "k": 4096, "r": 16, "l": 2, "s": 3},
        # a ragged middle size with an fp32 gradient
        {**back, "name": "back 333 rows f32", "m": 333, "n": 4096, "k": 11008, "r": 8, "l": 2, "s": 2, "out": "f32",
         "behind": 13},
        # a training batch through the frozen up projection alone
        {**back, "name": "back 2048 rows", "m": 2048, "n": 11008, "k": 4096, "r": 0, "l": 0, "s": 0},
        # one token's activations
        {"name": "checkpoint 1x4096", "op": "checkpoint", "m": 1, "k": 4096, "x": "bf16", "out": "bf16"},
        # a training batch in front of the down projection
        {"name": "checkpoint 4096x11008", "op": "checkpoint", "m": 4096, "k": 11008, "x": "bf16", "out": "bf16"},
        # the gradients of one adapter over a training batch
        {**grads, "name": "grads 4096 rows", "m": 4096, "n": 11008, "k": 4096, "r": 16, "l": 1, "s": 1},
        # several adapters trained at once, ragged, odd width, fp32 gradients
        {**grads, "name": "grads 601 rows f32", "m": 601, "n": 2050, "k": 2048, "r": 64, "l": 5, "s": 7, "dy": "f32",
         "none": 0.2, "behind": 11},
        # forward and backward of one layer of a training step
        {**lora, "name": "step 2048 rows", "op": "step", "m": 2048, "n": 4096, "k": 4096, "r": 16, "l": 1, "s": 1},
    ]


def log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "back", "back", "checkpoint", "grads", "step"])
    unit = rng.choice([32, 128, 128, 128, 256])  # K is a multiple of 32; model widths are mostly multiples of 128
    k = unit * max(1, log_between(rng, 256, 11008) // unit)
    x = rng.choice(["bf16", "bf16", "bf16", "f32"])
    out = x if op == "step" else rng.choice(["bf16", "bf16", "f32"])
    if op == "checkpoint":
        return {"op": op, "m": log_between(rng, 1, 4096), "k": k, "x": x, "out": rng.choice(["bf16", "f16", "f32"])}
    n = log_between(rng, 100, 11008)
    r = rng.choice([8, 8, 16, 16, 16, 32, 40, 64, 128])
    l = log_between(rng, 1, max(1, 512 // r))
    most = 4096 if op == "grads" else 10 ** 11 // (2 * n * k) + 1
    m = log_between(rng, 1, min(4096, most) if x == "bf16" else min(256, most))
    s = log_between(rng, 1, min(m, 64))
    none = rng.choice([0.0, 0.0, 0.2])
    behind = rng.choice([0, 0, min(5, m - s), (m - s) // 3])
    if op == "grads":
        return {"op": op, "m": m, "n": n, "k": k, "r": r, "l": l, "s": s, "x": x, "dy": rng.choice([x, x, "f32"]),
                "none": none, "behind": behind}
    g = rng.choice([v for v in (32, 64, 128, 128, 128, 256) if k % v == 0])
    if op == "back" and rng.random() < 0.4:
        r = l = s = behind = 0
        none = 0.0
    return {"op": op, "m": m, "n": n, "k": k, "g": g, "r": r, "l": l, "s": s, "x": x, "ab": rng.choice([x, x, "f32"]),
            "out": out, "sz": rng.choice(["f16", "f16", "f32"]), "none": none, "behind": behind}


def used_adapters(case):
    """Adapters that some row has, about."""
    s = case["s"] * (1 - case["none"])
    return case["l"] * (1 - (1 - 1 / case["l"]) ** s) if case["l"] else 0


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    ck = m * (k + 4 * math.ceil(k / BLOCK))
    if op == "checkpoint":
        return {"bytes": m * k * (SIZE[case["x"]] + SIZE[case["out"]]) + 2 * ck, "flops": 3 * m * k}
    n, r = case["n"], case["r"]
    rows = (m - case["behind"]) * (1 - case["none"])
    if op == "grads":
        return {"bytes": ck * rows / m + rows * (n * SIZE[case["dy"]] + 8 * r) + 4 * case["l"] * r * (n + k),
                "flops": 2 * rows * r * (n + k)}
    weights = n * (k / 2 + 2 * (k // case["g"]) * SIZE[case["sz"]])
    low = used_adapters(case) * r * (n + k) * SIZE[case["ab"]]
    flops = 2 * m * n * k + 2 * rows * r * (n + k)
    if op == "lora":
        return {"bytes": weights + low + m * (k * SIZE[case["x"]] + n * SIZE[case["out"]]), "flops": flops}
    if op == "back":
        return {"bytes": weights + low + m * (n * SIZE[case["x"]] + k * SIZE[case["out"]]) + 4 * rows * r, "flops": flops}
    # both directions, the checkpoint written and read, the adapters' gradients in their own type
    return {"bytes": 2 * weights + 3 * low + 2 * m * (n + k) * SIZE[case["x"]] + 2 * ck,
            "flops": 2 * flops + 2 * rows * r * (n + k)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def normal(gen, shape, sigma, dtype):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * sigma).to(dtype)


def heavy(x, gen):
    """5% of the channels twenty times as large, as in the activations of large models."""
    cols = torch.rand((x.shape[-1],), generator=gen, device=DEV) < 0.05
    return torch.where(cols, x * 20, x)


def segments(case, seed):
    """Bounds of the requests' rows (ragged, each with one at least) and their adapters (-1: none), on the host."""
    gen = torch.Generator().manual_seed(seed)
    rows, s = case["m"] - case["behind"], case["s"]
    cuts = torch.randperm(rows - 1, generator=gen)[:s - 1].sort().values + 1
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([rows])])
    which = torch.randint(0, case["l"], (s,), generator=gen)
    which = torch.where(torch.rand((s,), generator=gen) < case["none"], -1, which)
    return offsets.to(torch.int32), which.to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, m, k = case["op"], case["m"], case["k"]
    s = {"case": case}
    if op == "checkpoint":
        s["x"] = heavy(normal(gen, (m, k), 1.0, torch.float32), gen).to(DTYPES[case["x"]])
        return s
    n, r, l = case["n"], case["r"], case["l"]
    if l:
        offsets, which = segments(case, seed)
        s["offsets"], s["adapters"] = offsets.to(DEV), which.to(DEV)
        s["scaling"] = torch.rand((l,), generator=gen, device=DEV) + 0.5
    if op == "grads":
        real = row_adapters(s["offsets"], s["adapters"], m) >= 0
        x = heavy(normal(gen, (m, k), 1.0, torch.float32), gen).to(DTYPES[case["x"]])
        s["xq"], s["xs"] = checkpoint_codes(x)
        s["dy"] = normal(gen, (m, n), 1e-3, DTYPES[case["dy"]])
        s["u"] = normal(gen, (m, r), 1.0, torch.float32) * real.unsqueeze(1)
        s["v"] = normal(gen, (m, r), 1e-3, torch.float32) * real.unsqueeze(1)
        return s
    s["wq"], s["ws"], s["wz"] = int4_quantize(normal(gen, (n, k), 0.02, torch.float32), case["g"], DTYPES[case["sz"]])
    if l:
        s["a"] = normal(gen, (l, r, k), k ** -0.5, DTYPES[case["ab"]])
        s["b"] = normal(gen, (l, n, r), 0.02, DTYPES[case["ab"]])
    if op != "back":
        s["x"] = heavy(normal(gen, (m, k), 1.0, torch.float32), gen).to(DTYPES[case["x"]])
    if op != "lora":
        s["dy"] = normal(gen, (m, n), 1e-3, DTYPES[case["x"]])
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def int4_quantize(w, g, sz):
    """Asymmetric groups of g: scale = (max - min) / 15, zero-point, codes; two codes a byte, the even column low."""
    b = w.reshape(w.shape[0], -1, g)
    lo, hi = b.amin(-1), b.amax(-1)
    scale = ((hi - lo) / 15).to(sz)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    sf = scale.to(torch.float32)
    zero = (-lo / sf).round().clamp(0, 15)
    code = ((b / sf.unsqueeze(-1)) + zero.unsqueeze(-1)).round().clamp(0, 15).to(torch.uint8).reshape(w.shape)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale, zero.to(sz)


def int4_values(packed, scales, zeros):
    s, z = scales.to(torch.float32).unsqueeze(-1), zeros.to(torch.float32).unsqueeze(-1)
    q = torch.stack([packed & 15, packed >> 4], -1).to(torch.float32).reshape(*scales.shape, -1)
    return ((q - z) * s).reshape(packed.shape[0], -1)


def blocks(x):
    """Rows in blocks of 128 columns, the last one filled up with zeros."""
    k = x.shape[1]
    return torch.nn.functional.pad(x, (0, -k % BLOCK)).reshape(x.shape[0], -1, BLOCK)


def checkpoint_codes(x):
    """int8 codes [M, K] and float32 scales [M, blocks]; the quotient in 64 bits, since 32 would move it across a border."""
    b = blocks(x.to(torch.float32))
    scale = b.abs().amax(-1) / 127
    safe = torch.where(scale == 0, torch.ones_like(scale), scale)
    code = (b.double() / safe.unsqueeze(-1).double()).round().clamp(-127, 127) * (scale != 0).unsqueeze(-1)
    return code.to(torch.int8).reshape(x.shape[0], -1)[:, :x.shape[1]].contiguous(), scale


def checkpoint_values(xq, xs):
    return (blocks(xq.to(torch.float32)) * xs.unsqueeze(-1)).reshape(xq.shape[0], -1)[:, :xq.shape[1]]


def row_adapters(offsets, which, m):
    """The adapter of each row, -1 for rows that no request owns."""
    row = torch.arange(m, device=offsets.device)
    seg = (row.unsqueeze(1) >= offsets[1:]).sum(1)
    inside = (row >= offsets[0]) & (seg < which.shape[0])
    return torch.where(inside, which[seg.clamp(max=which.shape[0] - 1)].long(), -1)


def chosen(s, m):
    """[M, L, 1]: 1 for the row's adapter, 0 for the others."""
    which = row_adapters(s["offsets"], s["adapters"], m)
    return (which.unsqueeze(1) == torch.arange(s["case"]["l"], device=DEV)).to(torch.float32).unsqueeze(-1)


def into(x, a, s):
    """x A^T of every adapter in one product, all but the row's own set to zero, times its scaling: [M, L, R]."""
    l, r, k = a.shape
    wide = torch.matmul(x, a.to(torch.float32).reshape(l * r, k).t()).reshape(x.shape[0], l, r)
    return wide * chosen(s, x.shape[0]) * s["scaling"].view(1, l, 1)


def out_of(u, b):
    """u B^T, B [L, N, R]."""
    l, n, r = b.shape
    return torch.matmul(u.reshape(u.shape[0], l * r), b.to(torch.float32).transpose(1, 2).reshape(l * r, n))


def forward_plain(s):
    x = s["x"].to(torch.float32)
    u = into(x, s["a"], s)
    return torch.matmul(x, int4_values(s["wq"], s["ws"], s["wz"]).t()) + out_of(u, s["b"]), u


def back_plain(s):
    dy = s["dy"].to(torch.float32)
    dx = torch.matmul(dy, int4_values(s["wq"], s["ws"], s["wz"]))
    if not s["case"]["l"]:
        return dx, None
    v = into(dy, s["b"].transpose(1, 2), s)
    return dx + out_of(v, s["a"].transpose(1, 2)), v


def grads_plain(dy, xhat, u, v):
    """u, v [M, L, R], zero but for the row's adapter."""
    m, l, r = u.shape
    da = torch.matmul(v.reshape(m, l * r).t(), xhat).reshape(l, r, -1)
    db = torch.matmul(u.reshape(m, l * r).t(), dy.to(torch.float32)).reshape(l, r, -1).transpose(1, 2).contiguous()
    return da, db


def run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "checkpoint":
        return checkpoint_values(*checkpoint_codes(s["x"])).to(DTYPES[case["out"]])
    if op == "grads":
        one = chosen(s, case["m"])
        return grads_plain(s["dy"], checkpoint_values(s["xq"], s["xs"]), s["u"].unsqueeze(1) * one, s["v"].unsqueeze(1) * one)
    dt = DTYPES[case["out"]]
    if op == "lora":
        return forward_plain(s)[0].to(dt)
    if op == "back":
        dx, v = back_plain(s)
        return dx.to(dt) if v is None else (dx.to(dt), v.sum(1))
    y, u = forward_plain(s)
    dx, v = back_plain(s)
    da, db = grads_plain(s["dy"], checkpoint_values(*checkpoint_codes(s["x"])), u, v)
    return y.to(dt), dx.to(dt), da.to(s["a"].dtype), db.to(s["b"].dtype)


def run_own(s):
    import dequant_gemm_quantize_amd as w4
    case = s["case"]
    op = case["op"]
    if op == "checkpoint":
        return w4.dequant_checkpoint_int8(*w4.quantize_checkpoint_int8(s["x"]), out_dtype=DTYPES[case["out"]])
    if op == "grads":
        return w4.lora_grads(s["xq"], s["xs"], s["dy"], s["u"], s["v"], s["offsets"], s["adapters"], case["l"])
    weight = (s["wq"], s["ws"], s["wz"], case["g"])
    dt = DTYPES[case["out"]]
    if op == "back" and not case["l"]:
        return w4.w4a16_matmul_t(s["dy"], *weight, out_dtype=dt)
    adapter = (s["a"], s["b"], s["scaling"], s["offsets"], s["adapters"])
    if op == "lora":
        return w4.w4a16_lora_matmul(s["x"], *weight, *adapter, out_dtype=dt)
    if op == "back":
        v = s["dy"].new_zeros((case["m"], case["r"]), dtype=torch.float32)  # rows without an adapter stay zero
        return w4.w4a16_lora_matmul_t(s["dy"], *weight, *adapter, out_dtype=dt, v=v), v
    leaves = [s[t].detach().requires_grad_() for t in ("x", "a", "b")]
    y = w4.lora_linear(leaves[0], *weight, leaves[1], leaves[2], *adapter[2:])
    return (y.detach(), *torch.autograd.grad(y, leaves, s["dy"]))


def run(state):
    if own:
        return run_own(state)
    return run_plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op, m = case["op"], case["m"]
    if op == "checkpoint":
        return exact_checkpoint(s["x"])
    if op == "grads":
        xhat = s["xq"].double() * s["xs"].double().repeat_interleave(BLOCK, 1)[:, :case["k"]]
        return exact_grads(case, s, xhat, s["u"].double(), s["v"].double())
    w = exact_weight(case, s)
    parts = []
    if op != "back":
        x = s["x"].double()
        y, u = x @ w.t(), torch.zeros((m, case["r"]), dtype=torch.float64, device=DEV)
        for rows, i in exact_rows(s):
            u[rows] = float(s["scaling"][i]) * (x[rows] @ s["a"][i].double().t())
            y[rows] += u[rows] @ s["b"][i].double().t()
        if op == "lora":
            return y
        parts.append(y)
    dy = s["dy"].double()
    dx = dy @ w
    if not case["l"]:
        return dx
    v = torch.zeros((m, case["r"]), dtype=torch.float64, device=DEV)
    for rows, i in exact_rows(s):
        v[rows] = float(s["scaling"][i]) * (dy[rows] @ s["b"][i].double())
        dx[rows] += v[rows] @ s["a"][i].double()
    if op == "back":
        return dx, v
    return (y, dx, *exact_grads(case, s, exact_checkpoint(s["x"]), u, v))


def exact_rows(s):
    """(rows of a request, its adapter), requests without one left out."""
    bounds, which = s["offsets"].tolist(), s["adapters"].tolist()
    return [(slice(lo, hi), i) for lo, hi, i in zip(bounds, bounds[1:], which) if i >= 0]


def exact_grads(case, s, xhat, u, v):
    dy = s["dy"].double()
    da = torch.zeros((case["l"], case["r"], case["k"]), dtype=torch.float64, device=DEV)
    db = torch.zeros((case["l"], case["n"], case["r"]), dtype=torch.float64, device=DEV)
    for rows, i in exact_rows(s):
        da[i] += v[rows].t().contiguous() @ xhat[rows]
        db[i] += dy[rows].t().contiguous() @ u[rows]
    return da, db


def exact_weight(case, s):
    c = torch.empty((case["n"], case["k"]), dtype=torch.float64, device=DEV)
    c[:, 0::2] = (s["wq"] % 16).double()
    c[:, 1::2] = (s["wq"] // 16).double()
    return (c - s["wz"].double().repeat_interleave(case["g"], 1)) * s["ws"].double().repeat_interleave(case["g"], 1)


def exact_checkpoint(x):
    """The scale is a float32 by definition; everything after it in 64 bits."""
    xd = x.double()
    parts = []
    for c in range(0, x.shape[1], BLOCK):
        part = xd[:, c:c + BLOCK]
        scale = (part.abs().amax(1, keepdim=True) / 127).float().double()
        code = (part / scale.where(scale != 0, 1.0)).round().clamp(-127, 127)
        parts.append(code * scale)
    return torch.cat(parts, 1)
