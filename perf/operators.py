"""Cases of the 4-bit floating-point and the grouped products, each in a plain form and as the library's calls.

Four operators:
  roundtrip    quantize_mxfp4 then dequant_mxfp4: the values that the 4-bit codes and block scales stand for
  matmul       mxfp4_matmul: both operands in microscaled 4-bit floating point
  mx_grouped   mxfp4_grouped_matmul: the same by expert, rows sorted by expert, ragged sizes
  w4_grouped   w4a16_grouped_matmul: bf16 or fp32 activations, group-wise INT4 weights, by expert
"""
import math

import torch

own = False

DEV = "cuda"
# E2M1: sign bit, then the magnitudes of codes 0..7.
MAGNITUDES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
# x above (or at, where the lower code is odd) these borders rounds to the next magnitude
BORDERS = [(0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)]
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoded token's activations on their way to the matrix cores
        {"name": "roundtrip 1x4096", "op": "roundtrip", "n": 1, "k": 4096, "in": "bf16", "out": "bf16"},
        # a ragged batch of fp32 activations in front of the down projection
        {"name": "roundtrip 1003x11008 f32", "op": "roundtrip", "n": 1003, "k": 11008, "in": "f32", "out": "f32"},
        # weight preparation of the 70B-class projection
        {"name": "roundtrip 28672x8192", "op": "roundtrip", "n": 28672, "k": 8192, "in": "bf16", "out": "bf16"},
        # decode of one token, Llama-7B up projection
        {"name": "matmul 1x11008x4096", "op": "matmul", "m": 1, "n": 11008, "k": 4096, "out": "bf16"},
        # a small, odd decode batch on the down projection, fp32 result (a residual kept in fp32)
        {"name": "matmul 33x4096x11008 f32", "op": "matmul", "m": 33, "n": 4096, "k": 11008, "out": "f32"},
        # a chunk of a prompt on the 70B-class projection
        {"name": "matmul 512x28672x8192", "op": "matmul", "m": 512, "n": 28672, "k": 8192, "out": "bf16"},
        # prefill on the Llama-7B up projection
        {"name": "matmul 2048x11008x4096", "op": "matmul", "m": 2048, "n": 11008, "k": 4096, "out": "bf16"},
        # decode: eight tokens, two experts each, of many small experts; most experts get no row
        {"name": "mx_grouped 16 rows 64 experts", "op": "mx_grouped", "t": 16, "e": 64, "n": 2048, "k": 2048,
         "out": "bf16", "behind": 0},
        # prefill of a mixture of eight large experts
        {"name": "mx_grouped 4096 rows 8 experts", "op": "mx_grouped", "t": 4096, "e": 8, "n": 11008, "k": 4096,
         "out": "bf16", "behind": 0},
        # decode: one token, two of eight experts
        {"name": "w4_grouped 2 rows 8 experts", "op": "w4_grouped", "t": 2, "e": 8, "n": 11008, "k": 4096, "g": 128,
         "x": "bf16", "sz": "f16", "out": "bf16", "behind": 0},
        # a ragged middle size, odd widths, a padded batch (rows behind the last expert's), groups of 64
        {"name": "w4_grouped 777 rows 16 experts", "op": "w4_grouped", "t": 777, "e": 16, "n": 2050, "k": 2048, "g": 64,
         "x": "bf16", "sz": "f16", "out": "f32", "behind": 23},
        # prefill of a mixture of eight large experts
        {"name": "w4_grouped 4096 rows 8 experts", "op": "w4_grouped", "t": 4096, "e": 8, "n": 11008, "k": 4096, "g": 128,
         "x": "bf16", "sz": "f16", "out": "bf16", "behind": 0},
    ]


def log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["roundtrip", "matmul", "mx_grouped", "w4_grouped"])
    unit = rng.choice([32, 128, 128, 256, 256])  # K is a multiple of 32; model widths are mostly multiples of 128
    k = unit * max(1, log_between(rng, 256, 11008) // unit)
    out = rng.choice(["bf16", "bf16", "f32"])
    if op == "roundtrip":
        n = log_between(rng, 1, 28672)
        return {"op": op, "n": n, "k": k, "in": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f16", "f32"])}
    if op == "matmul":
        n = log_between(rng, 100, 28672)
        m = log_between(rng, 1, min(4096, 2 * 10 ** 11 // (2 * n * k) + 1))
        return {"op": op, "m": m, "n": n, "k": k, "out": out}
    e = log_between(rng, 2, 64)
    n = log_between(rng, 100, max(101, min(11008, 3 * 10 ** 8 // (e * k))))
    t = log_between(rng, 1, min(4096, 3 * 10 ** 11 // (2 * n * k) + 1))
    behind = rng.choice([0, 0, min(5, t - 1), t // 3])
    if op == "mx_grouped":
        return {"op": op, "t": t, "e": e, "n": n, "k": k, "out": out, "behind": behind}
    g = rng.choice([x for x in (32, 64, 128, 128, 128, 256) if k % x == 0])
    x = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if x == "f32":  # fp32 activations: small layers and checks
        t, out = min(t, 64), "f32"
        behind = min(behind, t - 1)
    return {"op": op, "t": t, "e": e, "n": n, "k": k, "g": g, "x": x, "sz": rng.choice(["f16", "f16", "f32"]),
            "out": out, "behind": behind}


def work(case):
    op, k = case["op"], case["k"]
    mx = k / 2 + k / 32  # bytes of a row in microscaled 4-bit floating point
    if op == "roundtrip":
        n = case["n"]
        return {"bytes": n * (k * SIZE[case["in"]] + mx + k * SIZE[case["out"]]), "flops": 3 * n * k}
    n = case["n"]
    if op == "matmul":
        m = case["m"]
        return {"bytes": (m + n) * mx + m * n * SIZE[case["out"]], "flops": 2 * m * n * k}
    t = case["t"] - case["behind"]
    experts = case["e"] * (1 - (1 - 1 / case["e"]) ** t)  # experts that get a row, about
    if op == "mx_grouped":
        read = t * mx + experts * n * mx
    else:
        read = t * k * SIZE[case["x"]] + experts * n * (k / 2 + 2 * (k // case["g"]) * SIZE[case["sz"]])
    return {"bytes": read + t * n * SIZE[case["out"]], "flops": 2 * t * n * k}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def normal(gen, shape, sigma, dtype):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * sigma).to(dtype)


def heavy(x, gen):
    """5% of the channels twenty times as large, as in the activations of large models."""
    cols = torch.rand((x.shape[-1],), generator=gen, device=DEV) < 0.05
    return torch.where(cols, x * 20, x)


def expert_sizes(case, seed):
    """Rows of each expert: popularity falls with a random rank, so that some experts get many rows and some none."""
    gen = torch.Generator().manual_seed(seed)
    t, e = case["t"] - case["behind"], case["e"]
    popular = (torch.randperm(e, generator=gen) + 1.0) ** -0.5
    chosen = torch.multinomial(popular, t, replacement=True, generator=gen) if t else torch.zeros(0, dtype=torch.int64)
    return torch.bincount(chosen, minlength=e)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, k, n = case["op"], case["k"], case["n"]
    s = {"case": case}
    if op == "roundtrip":
        s["w"] = heavy(normal(gen, (n, k), 1.0, DTYPES[case["in"]]), gen)
        return s
    if op == "matmul":
        s["xq"], s["xs"] = mx_quantize(heavy(normal(gen, (case["m"], k), 1.0, torch.float32), gen))
        s["wq"], s["ws"] = mx_quantize(normal(gen, (n, k), 0.02, torch.float32))
        return s
    t, e = case["t"], case["e"]
    sizes = expert_sizes(case, seed)
    s["cap"] = max(1, int(sizes.max()))  # the plain form's padded rows per expert
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).to(torch.int32).to(DEV)
    s["y"] = torch.zeros((t, n), dtype=DTYPES[case["out"]], device=DEV)
    x = heavy(normal(gen, (t, k), 1.0, torch.float32), gen)
    w = normal(gen, (e * n, k), 0.02, torch.float32)
    if op == "mx_grouped":
        s["xq"], s["xs"] = mx_quantize(x)
        wq, ws = mx_quantize(w)
        s["wq"], s["ws"] = wq.view(e, n, k // 2), ws.view(e, n, k // 32)
        return s
    s["x"] = x.to(DTYPES[case["x"]])
    wq, ws, wz = int4_quantize(w, case["g"], DTYPES[case["sz"]])
    s["wq"], s["ws"], s["wz"] = wq.view(e, n, k // 2), ws.view(e, n, -1), wz.view(e, n, -1)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def mx_split(x):
    """Codes (0..15, one a byte) and scale bytes of the rows of x, in blocks of 32."""
    b = x.to(torch.float32).reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    byte = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)  # the exponent field less E2M1's largest exponent
    v = b * pow2(127 - byte).unsqueeze(-1)  # exact: the byte is at most 252
    a = v.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for border, inclusive in BORDERS:  # seven comparisons
        code += (a >= border) if inclusive else (a > border)
    code += (b.view(torch.int32) < 0).to(torch.uint8) * 8
    return code.reshape(x.shape), byte.to(torch.uint8)


def pow2(e):
    """2^e in fp32 for whole e in -126..127."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def mx_quantize(x):
    code, byte = mx_split(x)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte


def nibbles(packed):
    return torch.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)


def mx_values(packed, scales):
    """The values in fp32: magnitude times 2^(byte - 127), exactly."""
    table = torch.tensor(MAGNITUDES + [-v for v in MAGNITUDES], dtype=torch.float32, device=packed.device)
    v = table[nibbles(packed).to(torch.int32)].reshape(*packed.shape[:-1], -1, 32)
    e = scales.to(torch.int32) - 127
    half = e // 2
    return (v * pow2(half).unsqueeze(-1) * pow2(e - half).unsqueeze(-1)).reshape(*packed.shape[:-1], -1)


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
    q = nibbles(packed).to(torch.float32).reshape(*scales.shape, -1)
    return ((q - z) * s).reshape(*packed.shape[:-1], -1)


def grouped_plain(x, w, offsets, cap, y):
    """Rows padded to the largest expert's count, one batched product, rows taken back out."""
    t = x.shape[0]
    start, stop = offsets[:-1].to(torch.int64), offsets[1:].to(torch.int64)
    rows = (start.unsqueeze(1) + torch.arange(cap, device=x.device)).clamp(max=t - 1)
    full = torch.bmm(x[rows], w.transpose(1, 2).contiguous())
    row = torch.arange(t, device=x.device)
    expert = (row.unsqueeze(1) >= stop).sum(1)
    real = expert < w.shape[0]
    expert = expert.clamp(max=w.shape[0] - 1)
    got = full[expert, (row - start[expert]).clamp(0, cap - 1)]
    y.copy_(torch.where(real.unsqueeze(1), got.to(y.dtype), y))
    return y


def run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "roundtrip":
        return mx_values(*mx_quantize(s["w"])).to(DTYPES[case["out"]])
    if op == "matmul":
        return torch.matmul(mx_values(s["xq"], s["xs"]), mx_values(s["wq"], s["ws"]).t()).to(DTYPES[case["out"]])
    if op == "mx_grouped":
        return grouped_plain(mx_values(s["xq"], s["xs"]), mx_values(s["wq"], s["ws"]), s["offsets"], s["cap"], s["y"])
    return grouped_plain(s["x"].to(torch.float32), int4_values(s["wq"], s["ws"], s["wz"]), s["offsets"], s["cap"], s["y"])


def run_own(s):
    import dequant_gemm_quantize_amd as w4
    case = s["case"]
    op = case["op"]
    if op == "roundtrip":
        return w4.dequant_mxfp4(*w4.quantize_mxfp4(s["w"]), out_dtype=DTYPES[case["out"]])
    if op == "matmul":
        return w4.mxfp4_matmul(s["xq"], s["xs"], s["wq"], s["ws"], out_dtype=DTYPES[case["out"]])
    if op == "mx_grouped":
        return w4.mxfp4_grouped_matmul(s["xq"], s["xs"], s["offsets"], s["wq"], s["ws"], out=s["y"])
    return w4.w4a16_grouped_matmul(s["x"], s["offsets"], s["wq"], s["ws"], s["wz"], case["g"], out=s["y"])


def run(state):
    if own:
        return run_own(state)
    return run_plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "roundtrip":
        return torch.cat([mx_exact_round(part.double()) for part in s["w"].split(1024)])
    if op == "matmul":
        x = mx_exact_values(s["xq"], s["xs"])
        return torch.cat([x @ mx_exact_values(q, b).t() for q, b in zip(s["wq"].split(2048), s["ws"].split(2048))], 1)
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    bounds = s["offsets"].tolist()
    for e in range(case["e"]):
        a, b = bounds[e], bounds[e + 1]
        if op == "mx_grouped":
            x, w = mx_exact_values(s["xq"][a:b], s["xs"][a:b]), mx_exact_values(s["wq"][e], s["ws"][e])
        else:
            x, w = s["x"][a:b].double(), int4_exact_values(s["wq"][e], s["ws"][e], s["wz"][e])
        y[a:b] = x @ w.t()
    return y


def exact_pow2(e):
    """2^e in 64 bits for whole e, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def mx_exact_round(x):
    """Nearest E2M1 multiple of 2^E, ties to the even code: steps of 1/2 below 2, 1 below 4, 2 above; at most 6."""
    b = x.reshape(x.shape[0], -1, 32)
    top = torch.frexp(b.abs().amax(-1, keepdim=True))
    exponent = torch.where(top.mantissa == 0, -127, top.exponent - 3).clamp(min=-127)
    v = b * exact_pow2(-exponent)
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()
    r = ((v / step).round() * step).clamp(-6, 6)
    return (r * exact_pow2(exponent)).reshape(x.shape)


def mx_exact_values(packed, scales):
    """sign, two exponent bits and one mantissa bit, read as such."""
    c = torch.empty((*packed.shape[:-1], packed.shape[-1] * 2), dtype=torch.float64, device=DEV)
    c[..., 0::2] = (packed % 16).double()
    c[..., 1::2] = (packed // 16).double()
    sign = 1 - 2 * (c >= 8).double()
    m = c % 8
    exponent, mantissa = (m / 2).floor(), m % 2
    v = torch.where(exponent == 0, mantissa / 2, (1 + mantissa / 2) * exact_pow2(exponent - 1))
    return sign * v * exact_pow2(scales.to(torch.int64) - 127).repeat_interleave(32, -1)


def int4_exact_values(packed, scales, zeros):
    c = torch.empty((packed.shape[0], packed.shape[1] * 2), dtype=torch.float64, device=DEV)
    c[:, 0::2] = (packed % 16).double()
    c[:, 1::2] = (packed // 16).double()
    g = c.shape[1] // scales.shape[1]
    return (c - zeros.double().repeat_interleave(g, 1)) * scales.double().repeat_interleave(g, 1)
