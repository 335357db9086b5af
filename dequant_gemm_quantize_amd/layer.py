"""PyTorch layer over the library: a drop-in for a bias-free nn.Linear whose
weight is stored as group-wise INT4 codes and multiplied by the fused
dequantize-matmul ("Building a From-Scratch Group-Wise INT4 Quantization
Layer for LLaMA Weights", Step 3: the quantized linear layer; Step 5: the
replacement pass over a model).

Every numeric step runs in the HIP kernels behind libw4.so: quantization at
construction (asymmetric, symmetric, symmetric with a percentile or MSE
calibrated scale, or GPTQ with calibration activations), the product in forward (W4A16, or W4A8 with per-token
INT8 activations).  This module only reshapes tensors and keeps the buffers.
Their weights are frozen.  Gradients pass a QuantizedLinear of bf16 or fp32
activations to its input, and LoRALinear trains low-rank adapters beside such a
weight; no gradient flows through the results of the layers that quantize
their activations (act_int8, MXFP4Linear) or of QuantizedExperts.
"""
from __future__ import annotations

from typing import Callable, Optional

import torch

from . import _lib

QUANTIZERS = {
    "asym": lambda w, g, sz, p: _lib.quantize_pack_int4(w, g, sz),
    "sym": lambda w, g, sz, p: _lib.quantize_pack_int4_sym(w, g, sz),
    "percentile": lambda w, g, sz, p: _lib.quantize_pack_int4_sym_percentile(w, g, 99.9 if p is None else p, sz),
    "mse": lambda w, g, sz, p: _lib.quantize_pack_int4_sym_mse(w, g, 1000 if p is None else int(p), sz),
    "gptq": lambda w, g, sz, p: _gptq(w, g, sz, p, False),
    "gptq_sym": lambda w, g, sz, p: _gptq(w, g, sz, p, True),
}


def _gptq(w: torch.Tensor, g: int, sz: torch.dtype, x: Optional[torch.Tensor], symmetric: bool):
    """GPTQ ([P4] Step 3) with calibration rows x [T, in_features] (float32,
    on the weight's GPU): Hessian, inverse Cholesky factor, column sweep."""
    if x is None:
        raise ValueError("GPTQ modes need the calibration rows X [T, in_features] as param")
    h = _lib.gptq_hessian(x.reshape(-1, x.shape[-1]).to(torch.float32).contiguous())
    u = _lib.gptq_inverse_cholesky(h, overwrite_h=True)
    # The sweep uses its weight argument as working storage.  A float32
    # contiguous weight converts to itself, so the sweep may take it over
    # only when the conversion made a copy; otherwise the wrapper copies it
    # and the caller's weight (possibly a tied parameter) is left unchanged.
    wf = w.to(torch.float32).contiguous()
    owned = wf.data_ptr() != w.data_ptr()
    return _lib.gptq_quantize_pack_int4(wf, u, g, symmetric, sz, overwrite_w=owned)


class _FrozenLinear(torch.autograd.Function):
    """y of w4a16_matmul, differentiable with respect to x: keeps the weight (not copied), nothing of x."""

    @staticmethod
    def forward(ctx, x, packed, scales, zeros, group_size, out_dtype):
        ctx.save_for_backward(packed, scales, zeros)
        ctx.group_size, ctx.dtype = group_size, x.dtype
        return _lib.w4a16_matmul(x, packed, scales, zeros, group_size, out_dtype=out_dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        dx = _lib.w4a16_matmul_t(_at_16_bytes(dy), *ctx.saved_tensors, ctx.group_size, out_dtype=ctx.dtype)
        return dx, None, None, None, None, None


class QuantizedLinear(torch.nn.Module):
    """y = x . dequant(Wq)^T with W [out_features, in_features] held as packed
    INT4 codes [N, K/2], scales and zero-points [N, K/g].

    forward(x): x [..., in_features] in bf16 or fp32 on the weight's GPU;
    returns [..., out_features] in ``out_dtype`` (default: x's dtype).  With
    ``act_int8=True`` the activations are quantized per token to INT8 first
    and the W4A8 product is used (bf16 output, which carries no gradient).

    Differentiable once with respect to x (w4a16_matmul_t; not with
    ``act_int8``); the weight is frozen."""

    def __init__(self, in_features: int, out_features: int, group_size: int = 128,
                 scale_dtype: torch.dtype = torch.float16, act_int8: bool = False,
                 out_dtype: Optional[torch.dtype] = None, device=None):
        super().__init__()
        if in_features % group_size or group_size % 32:
            raise ValueError("in_features must be a multiple of group_size, itself a multiple of 32")
        self.in_features = in_features
        self.out_features = out_features
        self.group_size = group_size
        self.act_int8 = act_int8
        self.out_dtype = out_dtype
        ng = in_features // group_size
        self.register_buffer("packed", torch.zeros((out_features, in_features // 2), dtype=torch.uint8,
                                                   device=device))
        self.register_buffer("scales", torch.ones((out_features, ng), dtype=scale_dtype, device=device))
        self.register_buffer("zeros", torch.zeros((out_features, ng), dtype=scale_dtype, device=device))

    @classmethod
    def from_weight(cls, weight: torch.Tensor, group_size: int = 128, mode: str = "asym",
                    param=None, scale_dtype: torch.dtype = torch.float16, act_int8: bool = False,
                    out_dtype: Optional[torch.dtype] = None) -> "QuantizedLinear":
        """Quantize W [out, in] (bf16 or fp32, on the GPU) with ``mode`` in
        asym / sym / percentile (param: p, default 99.9) / mse (param:
        candidates, default 1000) / gptq or gptq_sym (param: calibration
        rows X [T, in], required)."""
        if mode not in QUANTIZERS:
            raise ValueError(f"mode must be one of {sorted(QUANTIZERS)}")
        n, k = weight.shape
        layer = cls(k, n, group_size, scale_dtype, act_int8, out_dtype, device=weight.device)
        w = weight.detach()
        if w.dtype not in (torch.bfloat16, torch.float32):
            w = w.to(torch.float32)
        p, s, z = QUANTIZERS[mode](w.contiguous(), group_size, scale_dtype, param)
        layer.packed.copy_(p)
        layer.scales.copy_(s)
        layer.zeros.copy_(z)
        return layer

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, **kw) -> "QuantizedLinear":
        if linear.bias is not None:
            raise ValueError("QuantizedLinear has no bias; the linear layer has one")
        return cls.from_weight(linear.weight, **kw)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"x has {x.shape[-1]} features, the layer takes {self.in_features}")
        lead = x.shape[:-1]
        x2 = x.reshape(-1, self.in_features)
        if not x2.is_contiguous():
            x2 = x2.contiguous()
        if self.act_int8:
            xq, xs = _lib.quantize_act_int8(x2)
            y = _lib.w4a8_matmul(xq, xs, self.packed, self.scales, self.zeros, self.group_size,
                                 out_dtype=self.out_dtype or torch.bfloat16)
        else:
            args = (x2, self.packed, self.scales, self.zeros, self.group_size, self.out_dtype or x.dtype)
            y = _FrozenLinear.apply(*args) if x2.requires_grad and torch.is_grad_enabled() else _lib.w4a16_matmul(*args)
        return y.reshape(*lead, self.out_features)

    def dequantize(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """The dense weight (q - zp) * scale, for inspection."""
        return _lib.dequant_int4(self.packed, self.scales, self.zeros, self.group_size, out_dtype=dtype)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, "
                f"group_size={self.group_size}, act_int8={self.act_int8}")


def _float_weight(w: torch.Tensor) -> torch.Tensor:
    """A weight as the quantizers take it: bf16 or fp32, dense."""
    w = w.detach()
    return (w if w.dtype in (torch.bfloat16, torch.float32) else w.to(torch.float32)).contiguous()


def _activations(x2: torch.Tensor) -> torch.Tensor:
    """Activations as the kernels take them: fp16 ones in float32, which holds them."""
    return x2 if x2.dtype in (torch.bfloat16, torch.float32) else x2.to(torch.float32)


def _at_16_bytes(t: torch.Tensor) -> torch.Tensor:
    """t dense and at a 16-byte address, as the kernels take it.  A dense view into a larger tensor, as the backward
    of torch.cat makes them, may begin at any element."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


def _result_dtype(x: torch.Tensor, out_dtype: Optional[torch.dtype]) -> torch.dtype:
    return out_dtype or (x.dtype if x.is_floating_point() else torch.float32)


def _product_dtype(dt: torch.dtype) -> torch.dtype:
    """The type of y to ask a product for where the layer's result is of type dt (the products give fp32 and bf16)."""
    return torch.bfloat16 if dt == torch.bfloat16 else torch.float32


class MXFP4Linear(torch.nn.Module):
    """y = x . Wᵀ with both operands in microscaled 4-bit floating point
    (MXFP4): W [out_features, in_features] held as codes [N, K/2] and block
    scales [N, K/32], x quantized in forward, the product on the matrix
    cores' 4-bit inputs.

    forward(x): x [..., in_features] in bf16, fp32 or fp16 on the weight's
    GPU; returns [..., out_features] in ``out_dtype`` (default: x's dtype)."""

    def __init__(self, in_features: int, out_features: int, out_dtype: Optional[torch.dtype] = None, device=None):
        super().__init__()
        if in_features <= 0 or in_features % 32:
            raise ValueError("in_features must be a positive multiple of 32")
        self.in_features = in_features
        self.out_features = out_features
        self.out_dtype = out_dtype
        self.register_buffer("packed", torch.zeros((out_features, in_features // 2), dtype=torch.uint8, device=device))
        self.register_buffer("scales", torch.full((out_features, in_features // 32), 127, dtype=torch.uint8,
                                                  device=device))

    @classmethod
    def from_weight(cls, weight: torch.Tensor, out_dtype: Optional[torch.dtype] = None) -> "MXFP4Linear":
        n, k = weight.shape
        layer = cls(k, n, out_dtype, device=weight.device)
        _lib.quantize_mxfp4(_float_weight(weight), out=(layer.packed, layer.scales))
        return layer

    @classmethod
    def from_linear(cls, linear: torch.nn.Linear, **kw) -> "MXFP4Linear":
        if linear.bias is not None:
            raise ValueError("MXFP4Linear has no bias; the linear layer has one")
        return cls.from_weight(linear.weight, **kw)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"x has {x.shape[-1]} features, the layer takes {self.in_features}")
        xq, xs = _lib.quantize_mxfp4(_activations(x.reshape(-1, self.in_features).contiguous()))
        dt = _result_dtype(x, self.out_dtype)
        y = _lib.mxfp4_matmul(xq, xs, self.packed, self.scales, out_dtype=_product_dtype(dt)).to(dt)
        return y.reshape(*x.shape[:-1], self.out_features)

    def dequantize(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """The dense weight, for inspection."""
        return _lib.dequant_mxfp4(self.packed, self.scales, out_dtype=dtype)

    def extra_repr(self) -> str:
        return f"in_features={self.in_features}, out_features={self.out_features}"


class QuantizedExperts(torch.nn.Module):
    """The weights [experts, out_features, in_features] of one projection of a
    mixture of experts, in the INT4 format (``fmt="int4"``: W4A16 product) or
    in MXFP4 (``fmt="mxfp4"``: activations quantized in forward).

    forward(x, offsets): x [T, in_features] in bf16, fp32 or fp16 with its rows
    sorted by expert; offsets int32 [experts + 1] on the GPU, expert e owning
    rows offsets[e] .. offsets[e+1]-1; returns [T, out_features] in
    ``out_dtype`` (default: x's dtype), or ``out`` (fp32 or bf16).  Rows that no
    expert owns are not written (pass ``out`` to choose what they hold)."""

    def __init__(self, experts: int, in_features: int, out_features: int, fmt: str = "int4", group_size: int = 128,
                 scale_dtype: torch.dtype = torch.float16, out_dtype: Optional[torch.dtype] = None, device=None):
        super().__init__()
        if fmt not in ("int4", "mxfp4"):
            raise ValueError('fmt must be "int4" or "mxfp4"')
        self.experts, self.in_features, self.out_features = experts, in_features, out_features
        self.fmt, self.out_dtype = fmt, out_dtype
        self.group_size = group_size if fmt == "int4" else 32
        if in_features <= 0 or in_features % self.group_size or self.group_size % 32:
            raise ValueError("in_features must be a multiple of the group size, itself a multiple of 32")
        shape = (experts, out_features, in_features // self.group_size)
        self.register_buffer("packed", torch.zeros((experts, out_features, in_features // 2), dtype=torch.uint8,
                                                   device=device))
        if fmt == "int4":
            self.register_buffer("scales", torch.ones(shape, dtype=scale_dtype, device=device))
            self.register_buffer("zeros", torch.zeros(shape, dtype=scale_dtype, device=device))
        else:
            self.register_buffer("scales", torch.full(shape, 127, dtype=torch.uint8, device=device))

    @classmethod
    def from_weight(cls, weight: torch.Tensor, fmt: str = "int4", group_size: int = 128, mode: str = "asym",
                    scale_dtype: torch.dtype = torch.float16, out_dtype: Optional[torch.dtype] = None
                    ) -> "QuantizedExperts":
        """Quantize W [experts, out, in]; ``mode`` (INT4) is asym, sym,
        percentile or mse, as in QuantizedLinear.from_weight."""
        if weight.dim() != 3:
            raise ValueError("weight must be [experts, out, in]")
        if fmt == "int4" and mode not in ("asym", "sym", "percentile", "mse"):
            raise ValueError("mode must be asym, sym, percentile or mse")
        e, n, k = weight.shape
        layer = cls(e, k, n, fmt, group_size, scale_dtype, out_dtype, device=weight.device)
        w = _float_weight(weight).reshape(e * n, k)
        if fmt == "mxfp4":
            parts = zip((layer.packed, layer.scales), _lib.quantize_mxfp4(w))
        else:
            parts = zip((layer.packed, layer.scales, layer.zeros), QUANTIZERS[mode](w, group_size, scale_dtype, None))
        for buf, part in parts:
            buf.copy_(part.view(buf.shape))
        return layer

    def forward(self, x: torch.Tensor, offsets: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
        dt = _result_dtype(x, self.out_dtype)
        ask = _product_dtype(dt)
        x = _activations(x.contiguous())
        if self.fmt == "mxfp4":
            xq, xs = _lib.quantize_mxfp4(x)
            y = _lib.mxfp4_grouped_matmul(xq, xs, offsets, self.packed, self.scales, out_dtype=ask, out=out)
        else:
            y = _lib.w4a16_grouped_matmul(x, offsets, self.packed, self.scales, self.zeros, self.group_size,
                                          out_dtype=ask, out=out)
        return y if out is not None else y.to(dt)

    def dequantize(self, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
        """The dense weights [experts, out, in], for inspection."""
        flat = [b.view(-1, b.shape[-1]) for b in (self.packed, self.scales)]
        if self.fmt == "mxfp4":
            w = _lib.dequant_mxfp4(*flat, out_dtype=dtype)
        else:
            w = _lib.dequant_int4(*flat, self.zeros.view(-1, self.zeros.shape[-1]), self.group_size, out_dtype=dtype)
        return w.view(self.experts, self.out_features, self.in_features)

    def extra_repr(self) -> str:
        return (f"experts={self.experts}, in_features={self.in_features}, out_features={self.out_features}, "
                f"fmt={self.fmt}, group_size={self.group_size}")


class _LoRALinear(torch.autograd.Function):
    """y of w4a16_lora_matmul, differentiable with respect to x, a and b.  What
    is kept for the backward pass of x is its 8-bit checkpoint, and only if a or b is trained."""

    @staticmethod
    def forward(ctx, x, packed, scales, zeros, group_size, a, b, scaling, offsets, adapters):
        u = x.new_empty((x.shape[0], a.shape[1]), dtype=torch.float32)
        y = _lib.w4a16_lora_matmul(x, packed, scales, zeros, group_size, a, b, scaling, offsets, adapters, u=u)
        trained = ctx.needs_input_grad[5] or ctx.needs_input_grad[6]
        kept = (u, *_lib.quantize_checkpoint_int8(x)) if trained else ()
        ctx.save_for_backward(packed, scales, zeros, a, b, scaling, offsets, adapters, *kept)
        ctx.group_size = group_size
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        packed, scales, zeros, a, b, scaling, offsets, adapters, *kept = ctx.saved_tensors
        dy = _at_16_bytes(dy)
        v = dy.new_empty((dy.shape[0], a.shape[1]), dtype=torch.float32)
        dx = _lib.w4a16_lora_matmul_t(dy, packed, scales, zeros, ctx.group_size, a, b, scaling, offsets, adapters, v=v)
        da = db = None
        if kept:
            da, db = _lib.lora_grads(kept[1], kept[2], dy, kept[0], v, offsets, adapters, a.shape[0])
            da, db = da.to(a.dtype), db.to(b.dtype)
        return dx, None, None, None, None, da, db, None, None, None


def lora_linear(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, group_size: int,
                a: torch.Tensor, b: torch.Tensor, scaling: torch.Tensor, offsets: torch.Tensor,
                adapters: torch.Tensor) -> torch.Tensor:
    """w4a16_lora_matmul (arguments as there; y in x's dtype), differentiable
    once with respect to x, a and b; the INT4 weight stays frozen and scaling is a
    constant.  Between forward and backward it keeps the weight (not copied),
    u [M, R] and, if a or b needs a gradient, x in 8 bits: a's gradient is the one
    at the values that the checkpoint stands for, b's that of u from x itself."""
    args = (x, packed, scales, zeros, group_size, a, b, scaling, offsets, adapters)
    if torch.is_grad_enabled() and (x.requires_grad or a.requires_grad or b.requires_grad):
        return _LoRALinear.apply(*args)
    return _lib.w4a16_lora_matmul(*args)


class LoRALinear(torch.nn.Module):
    """y = x . dequant(Wq)^T + alpha / rank (x . A_l^T) . B_l^T: a frozen INT4
    projection with ``adapters`` trainable low-rank adapters beside it, one
    chosen per request.

    forward(x, offsets, which): x [..., in_features] in bf16, fp32 or fp16 on the
    weight's GPU, its rows (all leading dimensions taken together) in requests: rows
    offsets[s] .. offsets[s+1]-1 (int32 [S + 1] on the GPU) have adapter which[s]
    (int32 [S]; negative: none).  Without them every row has adapter 0.
    Returns [..., out_features] in x's dtype.

    Differentiable with respect to x and the parameters a [L, R, in] (normal,
    std 1 / sqrt(in)) and b [L, out, R] (zeros, so that a fresh adapter adds nothing);
    between forward and backward x is kept in 8 bits (quantize_checkpoint_int8).  The INT4 buffers are
    those of ``base``, not copies.  To capture a training step into a graph, run its
    warm-up on the capturing stream and let no earlier autograd graph of the same
    parameters live."""

    def __init__(self, base: QuantizedLinear, rank: int = 16, alpha: Optional[float] = None, adapters: int = 1,
                 dtype: torch.dtype = torch.float32):
        super().__init__()
        if rank <= 0 or rank % 8 or rank > 256:
            raise ValueError(f"rank = {rank} must be a multiple of 8 in 8 .. 256")
        if adapters < 1:
            raise ValueError(f"adapters = {adapters} must be at least 1")
        if dtype not in _lib.Y_DTYPES:
            raise ValueError(f"dtype must be float32 or bfloat16, got {dtype}")
        if base.act_int8:
            raise ValueError("LoRALinear multiplies bf16 or fp32 activations; base has act_int8")
        self.in_features, self.out_features, self.group_size = base.in_features, base.out_features, base.group_size
        self.rank, self.adapters = rank, adapters
        self.alpha = float(rank if alpha is None else alpha)
        dev = base.packed.device
        self.register_buffer("packed", base.packed)
        self.register_buffer("scales", base.scales)
        self.register_buffer("zeros", base.zeros)
        self.register_buffer("scaling", torch.full((adapters,), self.alpha / rank, dtype=torch.float32, device=dev))
        # one segment of all rows: (0, 1) times their number, and adapter 0
        self.register_buffer("_ends", torch.tensor([0, 1], dtype=torch.int32, device=dev), persistent=False)
        self.register_buffer("_first", torch.zeros((1,), dtype=torch.int32, device=dev), persistent=False)
        self.a = torch.nn.Parameter(torch.randn((adapters, rank, self.in_features), device=dev).mul_(
            self.in_features ** -0.5).to(dtype))
        self.b = torch.nn.Parameter(torch.zeros((adapters, self.out_features, rank), dtype=dtype, device=dev))

    def forward(self, x: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                which: Optional[torch.Tensor] = None) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"x has {x.shape[-1]} features, the layer takes {self.in_features}")
        if (offsets is None) != (which is None):
            raise ValueError("offsets and which come together")
        x2 = _at_16_bytes(_activations(x.reshape(-1, self.in_features)))
        if offsets is None:
            offsets, which = self._ends * x2.shape[0], self._first
        y = lora_linear(x2, self.packed, self.scales, self.zeros, self.group_size, _at_16_bytes(self.a),
                        _at_16_bytes(self.b), self.scaling, offsets, which)
        return y.to(_result_dtype(x, None)).reshape(*x.shape[:-1], self.out_features)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, out_features={self.out_features}, group_size={self.group_size}, "
                f"rank={self.rank}, alpha={self.alpha}, adapters={self.adapters}")


def replace_linears(module: torch.nn.Module, group_size: int = 128, mode: str = "asym",
                    skip: Optional[Callable[[str, torch.nn.Linear], bool]] = None, **kw) -> torch.nn.Module:
    """Replace, in place and recursively, every bias-free nn.Linear whose
    in_features is a multiple of group_size by a QuantizedLinear of its
    weight, or with ``mode="mxfp4"`` (groups of 32 whatever group_size says)
    by an MXFP4Linear.  ``skip(name, layer)`` can keep chosen layers dense."""
    unit = 32 if mode == "mxfp4" else group_size
    for name, child in list(module.named_children()):
        if isinstance(child, torch.nn.Linear):
            if child.bias is None and child.in_features % unit == 0 and not (skip and skip(name, child)):
                if mode == "mxfp4":
                    setattr(module, name, MXFP4Linear.from_linear(child, **kw))
                else:
                    setattr(module, name, QuantizedLinear.from_linear(child, group_size=group_size, mode=mode, **kw))
        else:
            replace_linears(child, group_size, mode, skip, **kw)
    return module
