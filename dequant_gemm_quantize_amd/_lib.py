"""ctypes binding of libw4.so.

Argument marshalling only: every computation runs in the HIP kernels behind
the C ABI declared in include/w4.h.  PyTorch supplies device memory and the
current stream.  There is no CPU fallback: if the library is missing or a
tensor is not on the GPU, the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Tuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("W4_LIB", os.path.join(HERE, "libw4.so"))

W4_F32, W4_F16, W4_BF16 = 0, 1, 2
W4_OK, W4_EINVAL, W4_EUNSUPPORTED, W4_EHIP = 0, -1, -2, -3

_DT = {torch.float32: W4_F32, torch.float16: W4_F16, torch.bfloat16: W4_BF16}

# (name, restype, argtypes) of every exported function, in header order.
_VP, _I, _I64, _I32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int32
SIGNATURES = [
    ("quantize_pack_int4", _I, [_VP, _I, _I64, _I64, _I32, _VP, _VP, _VP, _I, _VP]),
    ("quantize_pack_int4_sym", _I, [_VP, _I, _I64, _I64, _I32, _VP, _VP, _VP, _I, _VP]),
    ("quantize_pack_int4_sym_percentile", _I,
     [_VP, _I, _I64, _I64, _I32, ctypes.c_double, _VP, _VP, _VP, _I, _VP]),
    ("quantize_pack_int4_sym_mse", _I, [_VP, _I, _I64, _I64, _I32, _I32, _VP, _VP, _VP, _I, _VP]),
    ("dequant_int4", _I, [_VP, _VP, _VP, _I, _I64, _I64, _I32, _VP, _I, _VP]),
    ("quantize_act_int8", _I, [_VP, _I, _I64, _I64, _VP, _VP, _VP]),
    ("w4a16_matmul", _I, [_VP, _I, _I64, _I64, _VP, _VP, _VP, _I, _I64, _I32, _VP, _I, _VP]),
    ("w4a16_matmul_workspace_size", ctypes.c_size_t, [_I64, _I64, _I64, _I32, _I]),
    ("w4a16_matmul_ws", _I, [_VP, _I, _I64, _I64, _VP, _VP, _VP, _I, _I64, _I32, _VP, _I, _VP,
                             ctypes.c_size_t, _VP]),
    ("w4a16_matmul_noalloc", _I, [_VP, _I, _I64, _I64, _VP, _VP, _VP, _I, _I64, _I32, _VP, _I, _VP]),
    ("w4a8_matmul", _I, [_VP, _VP, _I64, _I64, _VP, _VP, _VP, _I, _I64, _I32, _VP, _I, _VP]),
    ("w4a8_matmul_workspace_size", ctypes.c_size_t, [_I64, _I64, _I64, _I32]),
    ("w4a8_matmul_ws", _I, [_VP, _VP, _I64, _I64, _VP, _VP, _VP, _I, _I64, _I32, _VP, _I, _VP,
                            ctypes.c_size_t, _VP]),
    ("gptq_hessian", _I, [_VP, _I64, _I64, _VP, _VP]),
    ("gptq_inverse_cholesky", _I, [_VP, _I64, _VP, _VP, _VP]),
    ("gptq_quantize_pack_int4", _I, [_VP, _VP, _I64, _I64, _I32, _I32, _VP, _VP, _VP, _I, _VP]),
    ("quantize_mxfp4", _I, [_VP, _I, _I64, _I64, _VP, _VP, _VP]),
    ("dequant_mxfp4", _I, [_VP, _VP, _I64, _I64, _VP, _I, _VP]),
    ("mxfp4_matmul", _I, [_VP, _VP, _I64, _I64, _VP, _VP, _I64, _VP, _I, _VP]),
    ("mxfp4_grouped_matmul", _I, [_VP, _VP, _I64, _I64, _VP, _I64, _VP, _VP, _I64, _VP, _I, _VP]),
    ("w4a16_grouped_matmul", _I, [_VP, _I, _I64, _I64, _VP, _I64, _VP, _VP, _VP, _I, _I64, _I32, _VP, _I, _VP]),
    ("quantize_checkpoint_int8", _I, [_VP, _I, _I64, _I64, _VP, _VP, _VP]),
    ("dequant_checkpoint_int8", _I, [_VP, _VP, _I64, _I64, _VP, _I, _VP]),
    ("w4a16_lora_matmul_workspace_size", ctypes.c_size_t, [_I64, _I64, _I64, _I32, _I, _I, _I]),
    ("w4a16_lora_matmul", _I, [_VP, _I, _I64, _I64, _VP, _VP, _VP, _I, _I64, _I32, _VP, _VP, _I, _I64, _I32, _VP, _VP,
                               _VP, _I64, _VP, _VP, _I, _VP, ctypes.c_size_t, _VP]),
    ("w4a16_matmul_t_workspace_size", ctypes.c_size_t, [_I64, _I64, _I64, _I32, _I, _I, _I]),
    ("w4a16_matmul_t", _I, [_VP, _I, _I64, _I64, _VP, _VP, _VP, _I, _I64, _I32, _VP, _I, _VP, ctypes.c_size_t, _VP]),
    ("w4a16_lora_matmul_t_workspace_size", ctypes.c_size_t, [_I64, _I64, _I64, _I32, _I, _I, _I, _I32, _I64]),
    ("w4a16_lora_matmul_t", _I, [_VP, _I, _I64, _I64, _VP, _VP, _VP, _I, _I64, _I32, _VP, _VP, _I, _I64, _I32, _VP,
                                 _VP, _VP, _I64, _VP, _VP, _I, _VP, ctypes.c_size_t, _VP]),
    ("lora_grads_workspace_size", ctypes.c_size_t, [_I64, _I64, _I64, _I, _I64, _I32]),
    ("lora_grads", _I, [_VP, _VP, _I64, _I64, _VP, _I, _I64, _VP, _VP, _VP, _VP, _I64, _I64, _I32, _VP, _VP, _VP,
                        ctypes.c_size_t, _VP]),
    ("w4_status_string", ctypes.c_char_p, [_I]),
    ("w4_last_error", ctypes.c_char_p, []),
    ("w4_version", ctypes.c_char_p, []),
]

_lib = None


class W4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libw4.so (once) and declare its signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(
            f"libw4.so not found at {p}: build it first "
            "(python -m dequant_gemm_quantize_amd.build or __graft_entry__.build())")
    lib = ctypes.CDLL(p)
    for name, res, args in SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _check(status: int) -> None:
    if status != W4_OK:
        lib = load()
        msg = lib.w4_last_error().decode() or lib.w4_status_string(status).decode()
        raise W4Error(status, msg)


def _ptr(t: torch.Tensor) -> int:
    return t.data_ptr()


def _gpu(*ts: torch.Tensor) -> torch.device:
    dev = None
    for t in ts:
        if not t.is_cuda:
            raise ValueError("libw4 runs on the GPU only: every tensor must be on a cuda (HIP) device")
        if not t.is_contiguous():
            raise ValueError("libw4 expects contiguous row-major tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("all tensors must be on the same device")
    return dev


def _stream(dev) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _dtype_code(dt: torch.dtype) -> int:
    if dt not in _DT:
        raise ValueError(f"unsupported dtype {dt}")
    return _DT[dt]


# Shape and dtype checks.  The C ABI sees only pointers and sizes, so a
# tensor of the wrong shape or dtype would be read or written out of bounds
# there; the wrappers, which know every tensor's size, refuse such calls
# before anything reaches the library.
def _expect(t: torch.Tensor, name: str, shape, dtypes) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        names = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} has dtype {str(t.dtype).replace('torch.', '')}, expected {names}")


def _matrix(t: torch.Tensor, name: str) -> Tuple[int, int]:
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor, got {t.dim()} dimensions")
    return int(t.shape[0]), int(t.shape[1])


def _ngroups(k: int, group_size: int) -> int:
    if group_size <= 0 or k % group_size:
        raise ValueError(f"K = {k} is not a multiple of group_size = {group_size}")
    return k // group_size


SZ_DTYPES = (torch.float16, torch.float32)


def _check_weights(packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, k: int,
                   group_size: int) -> int:
    """packed uint8 [N, K/2], scales and zeros [N, K/g] of one dtype; returns N."""
    n = _matrix(packed, "packed")[0]
    _expect(packed, "packed", (n, k // 2), (torch.uint8,))
    ng = _ngroups(k, group_size)
    _expect(scales, "scales", (n, ng), SZ_DTYPES)
    _expect(zeros, "zeros", (n, ng), (scales.dtype,))
    return n


# ---------------------------------------------------------------------------
# Public wrappers (same names as the C ABI)
# ---------------------------------------------------------------------------
def quantize_pack_int4(w: torch.Tensor, group_size: int, sz_dtype: torch.dtype = torch.float16,
                       out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None):
    """W [N, K] (fp32 or bf16) -> (packed uint8 [N, K/2], scales [N, K/g], zeros [N, K/g])."""
    return _quantize_pack(load().quantize_pack_int4, w, group_size, sz_dtype, out)


def quantize_pack_int4_sym(w: torch.Tensor, group_size: int, sz_dtype: torch.dtype = torch.float16,
                           out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None):
    """Symmetric variant: same arguments and outputs; every zero-point is 8."""
    return _quantize_pack(load().quantize_pack_int4_sym, w, group_size, sz_dtype, out)


def quantize_pack_int4_sym_percentile(w: torch.Tensor, group_size: int, percentile: float = 99.9,
                                      sz_dtype: torch.dtype = torch.float16,
                                      out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None):
    """Symmetric format, scale = (percentile of |w| per group) / 7."""
    fn = load().quantize_pack_int4_sym_percentile
    return _quantize_pack(lambda w_, d, n, k, g, *rest: fn(w_, d, n, k, g, float(percentile), *rest),
                          w, group_size, sz_dtype, out)


def quantize_pack_int4_sym_mse(w: torch.Tensor, group_size: int, candidates: int = 1000,
                               sz_dtype: torch.dtype = torch.float16,
                               out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None):
    """Symmetric format, step chosen per group by the MSE search over `candidates` steps."""
    fn = load().quantize_pack_int4_sym_mse
    return _quantize_pack(lambda w_, d, n, k, g, *rest: fn(w_, d, n, k, g, int(candidates), *rest),
                          w, group_size, sz_dtype, out)


def gptq_hessian(x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """H = X^T X / T + 1e-4 mean(diag) I (float64 [K, K]) from float32 calibration rows X [T, K]."""
    if x.dtype != torch.float32 or x.dim() != 2:
        raise ValueError("x must be a float32 [T, K] tensor")
    t, k = x.shape
    if out is not None:
        _expect(out, "out", (k, k), (torch.float64,))
    dev = _gpu(x)
    h = torch.empty((k, k), dtype=torch.float64, device=dev) if out is None else out
    _gpu(h)
    _check(load().gptq_hessian(_ptr(x), t, k, _ptr(h), _stream(dev)))
    return h


def gptq_inverse_cholesky(h: torch.Tensor, out: Optional[torch.Tensor] = None, overwrite_h: bool = False,
                          check: bool = True):
    """U (float64 [K, K], upper triangular, U^T U = H^-1).  h is used as the
    factorization's workspace: it is copied first unless overwrite_h.  With
    check, waits for the device status and raises if H is not positive
    definite; otherwise returns (u, info) with info a device int32 tensor."""
    if h.dtype != torch.float64 or h.dim() != 2 or h.shape[0] != h.shape[1]:
        raise ValueError("h must be a square float64 tensor")
    k = h.shape[0]
    if out is not None:
        _expect(out, "out", (k, k), (torch.float64,))
    dev = _gpu(h)
    work = h if overwrite_h else h.clone()
    u = torch.empty((k, k), dtype=torch.float64, device=dev) if out is None else out
    _gpu(u)
    info = torch.empty((1,), dtype=torch.int32, device=dev)
    _check(load().gptq_inverse_cholesky(_ptr(work), k, _ptr(u), _ptr(info), _stream(dev)))
    if not check:
        return u, info
    bad = int(info.item())
    if bad:
        raise ValueError(f"gptq_inverse_cholesky: H is not positive definite (pivot of column {bad - 1})")
    return u


def gptq_quantize_pack_int4(w: torch.Tensor, u: torch.Tensor, group_size: int, symmetric: bool = False,
                            sz_dtype: torch.dtype = torch.float16, overwrite_w: bool = False,
                            out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None):
    """GPTQ column sweep of W [N, K] (float32) with U from gptq_inverse_cholesky;
    returns (packed, scales, zeros) in the library's format.  W is copied
    first unless overwrite_w (the sweep uses it as working storage)."""
    if w.dtype != torch.float32 or w.dim() != 2:
        raise ValueError("w must be a float32 [N, K] tensor")
    if u.dtype != torch.float64 or tuple(u.shape) != (w.shape[1], w.shape[1]):
        raise ValueError("u must be a float64 [K, K] tensor")
    n, k = w.shape
    ng = _ngroups(k, group_size)
    if out is not None:
        _check_out3(out, n, k, ng)
    dev = _gpu(w, u)
    work = w if overwrite_w else w.clone()
    if out is None:
        packed = torch.empty((n, k // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((n, k // group_size), dtype=sz_dtype, device=dev)
        zeros = torch.empty((n, k // group_size), dtype=sz_dtype, device=dev)
    else:
        packed, scales, zeros = out
        _gpu(packed, scales, zeros)
    _check(load().gptq_quantize_pack_int4(_ptr(work), _ptr(u), n, k, group_size, int(bool(symmetric)),
                                          _ptr(packed), _ptr(scales), _ptr(zeros),
                                          _dtype_code(scales.dtype), _stream(dev)))
    return packed, scales, zeros


def _check_out3(out, n: int, k: int, ng: int) -> None:
    packed, scales, zeros = out
    _expect(packed, "packed", (n, k // 2), (torch.uint8,))
    _expect(scales, "scales", (n, ng), SZ_DTYPES)
    _expect(zeros, "zeros", (n, ng), (scales.dtype,))


def _quantize_pack(fn, w, group_size, sz_dtype, out):
    n, k = _matrix(w, "w")
    if w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"w has dtype {w.dtype}, expected float32 or bfloat16")
    ng = _ngroups(k, group_size)
    if out is not None:
        _check_out3(out, n, k, ng)
    elif sz_dtype not in SZ_DTYPES:
        raise ValueError(f"sz_dtype must be float16 or float32, got {sz_dtype}")
    dev = _gpu(w)
    if out is None:
        packed = torch.empty((n, k // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((n, k // group_size), dtype=sz_dtype, device=dev)
        zeros = torch.empty((n, k // group_size), dtype=sz_dtype, device=dev)
    else:
        packed, scales, zeros = out
        _gpu(packed, scales, zeros)
    _check(fn(_ptr(w), _dtype_code(w.dtype), n, k, group_size, _ptr(packed), _ptr(scales),
              _ptr(zeros), _dtype_code(scales.dtype), _stream(dev)))
    return packed, scales, zeros


def dequant_int4(packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, group_size: int,
                 out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None):
    """(packed, scales, zeros) -> dequantized W [N, K] in out_dtype."""
    lib = load()
    n, half = _matrix(packed, "packed")
    k = 2 * half
    _check_weights(packed, scales, zeros, k, group_size)
    if out is not None:
        _expect(out, "out", (n, k), tuple(_DT))
    dev = _gpu(packed, scales, zeros)
    w = torch.empty((n, k), dtype=out_dtype, device=dev) if out is None else out
    _gpu(w)
    _check(lib.dequant_int4(_ptr(packed), _ptr(scales), _ptr(zeros), _dtype_code(scales.dtype), n, k,
                            group_size, _ptr(w), _dtype_code(w.dtype), _stream(dev)))
    return w


def quantize_act_int8(x: torch.Tensor, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """x [M, K] (fp32 or bf16) -> (xq int8 [M, K], x_scale float32 [M])."""
    lib = load()
    m, k = _matrix(x, "x")
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"x has dtype {x.dtype}, expected float32 or bfloat16")
    if out is not None:
        _expect(out[0], "xq", (m, k), (torch.int8,))
        _expect(out[1], "x_scale", (m,), (torch.float32,))
    dev = _gpu(x)
    if out is None:
        xq = torch.empty((m, k), dtype=torch.int8, device=dev)
        xs = torch.empty((m,), dtype=torch.float32, device=dev)
    else:
        xq, xs = out
        _gpu(xq, xs)
    _check(lib.quantize_act_int8(_ptr(x), _dtype_code(x.dtype), m, k, _ptr(xq), _ptr(xs), _stream(dev)))
    return xq, xs


def w4a16_matmul_workspace_size(m: int, k: int, n: int, group_size: int,
                                x_dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace with which w4a16_matmul splits K for this shape (0: none)."""
    return int(load().w4a16_matmul_workspace_size(m, k, n, group_size, _dtype_code(x_dtype)))


def w4a16_matmul(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                 group_size: int, out_dtype: Optional[torch.dtype] = None,
                 out: Optional[torch.Tensor] = None, workspace="auto"):
    """y [M, N] = x [M, K] . dequant(W)^T; out_dtype defaults to x's dtype.

    workspace: "auto" (default) allocates, through torch, the workspace the
    library asks for on this shape (none for most shapes) and calls
    w4a16_matmul_ws; a uint8 device tensor is used as given; None calls
    w4a16_matmul, which uses none."""
    lib = load()
    m, k = _matrix(x, "x")
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"x has dtype {x.dtype}, expected float32 or bfloat16")
    if _matrix(packed, "packed")[1] * 2 != k:
        raise ValueError(f"packed has {packed.shape[1] * 2} columns of codes, x has K={k}")
    n = _check_weights(packed, scales, zeros, k, group_size)
    if out is not None:
        _expect(out, "out", (m, n), (torch.float32, torch.bfloat16))
    dev = _gpu(x, packed, scales, zeros)
    y = torch.empty((m, n), dtype=out_dtype or x.dtype, device=dev) if out is None else out
    _gpu(y)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be "auto", None or a uint8 tensor')
        nbytes = int(lib.w4a16_matmul_workspace_size(m, k, n, group_size, _dtype_code(x.dtype)))
        workspace = torch.empty((nbytes,), dtype=torch.uint8, device=dev) if nbytes else None
    args = (_ptr(x), _dtype_code(x.dtype), m, k, _ptr(packed), _ptr(scales), _ptr(zeros),
            _dtype_code(scales.dtype), n, group_size, _ptr(y), _dtype_code(y.dtype))
    if workspace is None:
        _check(lib.w4a16_matmul(*args, _stream(dev)))
    else:
        if workspace.dtype != torch.uint8 or workspace.dim() != 1:
            raise ValueError("workspace must be a 1-D uint8 tensor")
        _gpu(workspace)
        _check(lib.w4a16_matmul_ws(*args, _ptr(workspace), workspace.numel(), _stream(dev)))
    return y


def w4a8_matmul_workspace_size(m: int, k: int, n: int, group_size: int) -> int:
    """Bytes of workspace with which w4a8_matmul splits K for this shape (0: none)."""
    return int(load().w4a8_matmul_workspace_size(m, k, n, group_size))


def w4a8_matmul(xq: torch.Tensor, x_scale: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                zeros: torch.Tensor, group_size: int, out_dtype: torch.dtype = torch.bfloat16,
                out: Optional[torch.Tensor] = None, workspace="auto"):
    """y [M, N] = x_scale[m] * (xq [M, K] . dequant(W)^T).

    workspace: "auto" (default) allocates, through torch, the workspace the
    library asks for on this shape (none for most shapes) and calls
    w4a8_matmul_ws; a uint8 device tensor is used as given; None calls
    w4a8_matmul, which uses none."""
    lib = load()
    m, k = _matrix(xq, "xq")
    _expect(xq, "xq", (m, k), (torch.int8,))
    _expect(x_scale, "x_scale", (m,), (torch.float32,))
    if _matrix(packed, "packed")[1] * 2 != k:
        raise ValueError(f"packed has {packed.shape[1] * 2} columns of codes, xq has K={k}")
    n = _check_weights(packed, scales, zeros, k, group_size)
    if out is not None:
        _expect(out, "out", (m, n), (torch.float32, torch.bfloat16))
    dev = _gpu(xq, x_scale, packed, scales, zeros)
    y = torch.empty((m, n), dtype=out_dtype, device=dev) if out is None else out
    _gpu(y)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('workspace must be "auto", None or a uint8 tensor')
        nbytes = int(lib.w4a8_matmul_workspace_size(m, k, n, group_size))
        workspace = torch.empty((nbytes,), dtype=torch.uint8, device=dev) if nbytes else None
    args = (_ptr(xq), _ptr(x_scale), m, k, _ptr(packed), _ptr(scales), _ptr(zeros),
            _dtype_code(scales.dtype), n, group_size, _ptr(y), _dtype_code(y.dtype))
    if workspace is None:
        _check(lib.w4a8_matmul(*args, _stream(dev)))
    else:
        if workspace.dtype != torch.uint8 or workspace.dim() != 1:
            raise ValueError("workspace must be a 1-D uint8 tensor")
        _gpu(workspace)
        _check(lib.w4a8_matmul_ws(*args, _ptr(workspace), workspace.numel(), _stream(dev)))
    return y


# ---------------------------------------------------------------------------
# Microscaled 4-bit floating point and the products by expert
# ---------------------------------------------------------------------------
# A product of one token takes less time than these wrappers can: what follows
# asks each tensor as little as the checks need, looks for the words of an error
# only when there is one, and takes the current stream's handle (an int) without
# the Stream object around it (0.06 us against 1.06) where torch has that query,
# a private name.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _stream


def _device(*ts: torch.Tensor) -> int:
    """The index of the GPU that holds every one of the (dense) tensors."""
    dev = ts[0].get_device()
    for t in ts:
        if dev < 0 or t.get_device() != dev or not t.is_contiguous():
            _gpu(*ts)  # raises, with the reason
    return dev


def _launch(dev: int, fn, *args) -> None:
    """Call fn with dev's current stream, on dev whichever device is current."""
    if torch.cuda.current_device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status != W4_OK:
        _check(status)


def _mx_blocks(k: int) -> int:
    if k <= 0 or k % 32:
        raise ValueError(f"K = {k} is not a positive multiple of 32")
    return k // 32


def _check_mx(packed: torch.Tensor, scales: torch.Tensor, names: Tuple[str, str], lead: int) -> Tuple[int, ...]:
    """packed uint8 [..., K/2] and scales uint8 [..., K/32] of `lead` leading dimensions; returns (..., K)."""
    shape = packed.shape
    if len(shape) != lead + 1:
        raise ValueError(f"{names[0]} must be a {lead + 1}-D tensor, got {len(shape)} dimensions")
    k = 2 * shape[-1]
    if packed.dtype is not torch.uint8:
        _expect(packed, names[0], shape, (torch.uint8,))
    if scales.dtype is not torch.uint8 or scales.shape != (*shape[:-1], _mx_blocks(k)):
        _expect(scales, names[1], (*shape[:-1], _mx_blocks(k)), (torch.uint8,))
    return (*shape[:-1], k)


Y_DTYPES = (torch.float32, torch.bfloat16)


def _y_out(out: Optional[torch.Tensor], out_dtype: torch.dtype, shape, like: torch.Tensor) -> torch.Tensor:
    """out (checked by the caller against the other tensors' device), or a new tensor beside `like`."""
    if out is None:
        if out_dtype not in Y_DTYPES:
            raise ValueError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
        return like.new_empty(shape, dtype=out_dtype)
    _expect(out, "out", shape, Y_DTYPES)
    return out


def quantize_mxfp4(w: torch.Tensor, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """W or x [N, K] (fp32 or bf16) -> (packed uint8 [N, K/2], scales uint8 [N, K/32])."""
    n, k = _matrix(w, "w")
    if w.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"w has dtype {w.dtype}, expected float32 or bfloat16")
    nb = _mx_blocks(k)
    if out is not None:
        _expect(out[0], "packed", (n, k // 2), (torch.uint8,))
        _expect(out[1], "scales", (n, nb), (torch.uint8,))
        dev = _device(w, *out)
        packed, scales = out
    else:
        dev = _device(w)
        packed, scales = w.new_empty((n, k // 2), dtype=torch.uint8), w.new_empty((n, nb), dtype=torch.uint8)
    _launch(dev, load().quantize_mxfp4, _ptr(w), _dtype_code(w.dtype), n, k, _ptr(packed), _ptr(scales))
    return packed, scales


def dequant_mxfp4(packed: torch.Tensor, scales: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                  out: Optional[torch.Tensor] = None):
    """(packed, scales) -> the values [N, K] in out_dtype."""
    n, k = _check_mx(packed, scales, ("packed", "scales"), 1)
    if out is not None:
        _expect(out, "out", (n, k), tuple(_DT))
        dev = _device(packed, scales, out)
        w = out
    else:
        _dtype_code(out_dtype)
        dev = _device(packed, scales)
        w = packed.new_empty((n, k), dtype=out_dtype)
    _launch(dev, load().dequant_mxfp4, _ptr(packed), _ptr(scales), n, k, _ptr(w), _dtype_code(w.dtype))
    return w


def mxfp4_matmul(xq: torch.Tensor, xs: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                 out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None):
    """y [M, N] = dequant(xq) . dequant(W)^T, both operands from quantize_mxfp4."""
    m, k = _check_mx(xq, xs, ("xq", "xs"), 1)
    n, kw = _check_mx(packed, scales, ("packed", "scales"), 1)
    if kw != k:
        raise ValueError(f"packed has {kw} columns of codes, xq has K={k}")
    dev = _device(xq, xs, packed, scales) if out is None else _device(xq, xs, packed, scales, out)
    y = _y_out(out, out_dtype, (m, n), xq)
    _launch(dev, load().mxfp4_matmul, _ptr(xq), _ptr(xs), m, k, _ptr(packed), _ptr(scales), n, _ptr(y),
            _dtype_code(y.dtype))
    return y


def mxfp4_grouped_matmul(xq: torch.Tensor, xs: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor,
                         scales: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                         out: Optional[torch.Tensor] = None):
    """y [T, N]: rows offsets[e] .. offsets[e+1]-1 of x times expert e's W^T.

    xq uint8 [T, K/2] and xs [T, K/32]; packed [E, N, K/2] and scales
    [E, N, K/32]; offsets int32 [E + 1], rising, on the GPU (never read on the
    host).  Rows that no expert owns are not written: without out= they hold
    whatever the new tensor held."""
    t, k = _check_mx(xq, xs, ("xq", "xs"), 1)
    e, n, kw = _check_mx(packed, scales, ("packed", "scales"), 2)
    if kw != k:
        raise ValueError(f"packed has {kw} columns of codes, xq has K={k}")
    _expect(offsets, "offsets", (e + 1,), (torch.int32,))
    dev = _device(xq, xs, offsets, packed, scales) if out is None else _device(xq, xs, offsets, packed, scales, out)
    y = _y_out(out, out_dtype, (t, n), xq)
    _launch(dev, load().mxfp4_grouped_matmul, _ptr(xq), _ptr(xs), t, k, _ptr(offsets), e, _ptr(packed),
            _ptr(scales), n, _ptr(y), _dtype_code(y.dtype))
    return y


def w4a16_grouped_matmul(x: torch.Tensor, offsets: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
                         zeros: torch.Tensor, group_size: int, out_dtype: Optional[torch.dtype] = None,
                         out: Optional[torch.Tensor] = None):
    """y [T, N]: rows offsets[e] .. offsets[e+1]-1 of x [T, K] (bf16 or fp32)
    times expert e's dequant(W)^T; out_dtype defaults to x's dtype.

    packed [E, N, K/2], scales and zeros [E, N, K/g] in the INT4 format;
    offsets int32 [E + 1], rising, on the GPU (never read on the host).  Rows
    that no expert owns are not written: without out= they hold whatever the
    new tensor held."""
    t, k = _matrix(x, "x")
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"x has dtype {x.dtype}, expected float32 or bfloat16")
    if packed.dim() != 3:
        raise ValueError(f"packed must be a 3-D tensor, got {packed.dim()} dimensions")
    e, n = int(packed.shape[0]), int(packed.shape[1])
    _expect(packed, "packed", (e, n, k // 2), (torch.uint8,))
    ng = _ngroups(k, group_size)
    _expect(scales, "scales", (e, n, ng), SZ_DTYPES)
    _expect(zeros, "zeros", (e, n, ng), (scales.dtype,))
    _expect(offsets, "offsets", (e + 1,), (torch.int32,))
    dev = _device(x, offsets, packed, scales, zeros) if out is None else _device(x, offsets, packed, scales, zeros, out)
    y = _y_out(out, out_dtype or x.dtype, (t, n), x)
    _launch(dev, load().w4a16_grouped_matmul, _ptr(x), _dtype_code(x.dtype), t, k, _ptr(offsets), e, _ptr(packed),
            _ptr(scales), _ptr(zeros), _dtype_code(scales.dtype), n, group_size, _ptr(y), _dtype_code(y.dtype))
    return y


# ---------------------------------------------------------------------------
# Activation checkpoints in 8 bits, the transposed product, low-rank adapters
# ---------------------------------------------------------------------------
CHECKPOINT_BLOCK = 128  # columns of a block of the 8-bit checkpoint


def _checkpoint_blocks(k: int) -> int:
    if k <= 0 or k % 32:
        raise ValueError(f"K = {k} is not a positive multiple of 32")
    return -(-k // CHECKPOINT_BLOCK)


def quantize_checkpoint_int8(x: torch.Tensor, out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """x [M, K] (fp32 or bf16) -> (xq int8 [M, K], xs float32 [M, ceil(K/128)]), a scale for each 128 columns of a row."""
    m, k = _matrix(x, "x")
    if x.dtype not in Y_DTYPES:
        raise ValueError(f"x has dtype {x.dtype}, expected float32 or bfloat16")
    nb = _checkpoint_blocks(k)
    if out is not None:
        xq, xs = out
        _expect(xq, "xq", (m, k), (torch.int8,))
        _expect(xs, "xs", (m, nb), (torch.float32,))
        dev = _device(x, xq, xs)
    else:
        dev = _device(x)
        xq, xs = x.new_empty((m, k), dtype=torch.int8), x.new_empty((m, nb), dtype=torch.float32)
    _launch(dev, load().quantize_checkpoint_int8, _ptr(x), _dtype_code(x.dtype), m, k, _ptr(xq), _ptr(xs))
    return xq, xs


def _check_checkpoint(xq: torch.Tensor, xs: torch.Tensor) -> Tuple[int, int]:
    m, k = _matrix(xq, "xq")
    _expect(xq, "xq", (m, k), (torch.int8,))
    _expect(xs, "xs", (m, _checkpoint_blocks(k)), (torch.float32,))
    return m, k


def dequant_checkpoint_int8(xq: torch.Tensor, xs: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                            out: Optional[torch.Tensor] = None):
    """(xq, xs) -> the values [M, K] in out_dtype (fp32, fp16 or bf16)."""
    m, k = _check_checkpoint(xq, xs)
    if out is not None:
        _expect(out, "out", (m, k), tuple(_DT))
        dev = _device(xq, xs, out)
    else:
        _dtype_code(out_dtype)
        dev = _device(xq, xs)
        out = xq.new_empty((m, k), dtype=out_dtype)
    _launch(dev, load().dequant_checkpoint_int8, _ptr(xq), _ptr(xs), m, k, _ptr(out), _dtype_code(out.dtype))
    return out


# The wrappers of these products ask each tensor's shape and type once, look for
# the words of an error (the _expect calls) only behind a comparison that
# failed, and keep the workspaces' sizes, which depend on the arguments alone.
def _check_segments(offsets: torch.Tensor, adapters: torch.Tensor) -> int:
    """offsets int32 [S + 1] and adapters int32 [S]; returns S."""
    if adapters.dim() != 1:
        raise ValueError(f"adapters must be a 1-D tensor, got {adapters.dim()} dimensions")
    s = adapters.shape[0]
    if adapters.dtype is not torch.int32 or offsets.dtype is not torch.int32 or offsets.shape != (s + 1,):
        _expect(adapters, "adapters", (s,), (torch.int32,))
        _expect(offsets, "offsets", (s + 1,), (torch.int32,))
    return s


def _check_lora(a, b, scaling, offsets, adapters, k: int, n: int) -> Tuple[int, int, int]:
    """a [L, R, K] and b [L, N, R] of one dtype, scaling float32 [L], and the segments; returns (L, R, S)."""
    if a.dim() != 3:
        raise ValueError(f"a must be a 3-D tensor, got {a.dim()} dimensions")
    count, rank, width = a.shape
    dt = a.dtype
    if width != k or (dt is not torch.bfloat16 and dt is not torch.float32):
        _expect(a, "a", (count, rank, k), Y_DTYPES)
    if b.dtype is not dt or b.shape != (count, n, rank):
        _expect(b, "b", (count, n, rank), (dt,))
    if scaling.dtype is not torch.float32 or scaling.shape != (count,):
        _expect(scaling, "scaling", (count,), (torch.float32,))
    return count, rank, _check_segments(offsets, adapters)


def _int4_product(x, name: str, packed, scales, zeros, group_size: int, transposed: bool) -> Tuple[int, int, int]:
    """x [M, K] (or dy [M, N]) against an INT4 weight; returns (M, K, N)."""
    if x.dim() != 2 or packed.dim() != 2:
        _matrix(x, name), _matrix(packed, "packed")
    if x.dtype is not torch.bfloat16 and x.dtype is not torch.float32:
        raise ValueError(f"{name} has dtype {x.dtype}, expected float32 or bfloat16")
    m, d = x.shape
    n, half = packed.shape
    k = 2 * half
    groups = (n, _ngroups(k, group_size))
    if (packed.dtype is not torch.uint8 or scales.shape != groups or zeros.shape != groups
            or scales.dtype not in SZ_DTYPES or zeros.dtype is not scales.dtype):
        _check_weights(packed, scales, zeros, k, group_size)
    if d != (n if transposed else k):
        raise ValueError(f"{name} has {d} columns, the weight [N, K] is [{n}, {k}]")
    return m, k, n


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(name: str, *args) -> int:
    return int(getattr(load(), name)(*args))


def _given(out, shape, low, name: str, m: int, rank: int) -> tuple:
    """The caller's tensors for the result and for the rows' low-rank values, checked."""
    if out is not None:
        _expect(out, "out", shape, Y_DTYPES)
    if low is not None and (low.dtype is not torch.float32 or low.shape != (m, rank)):
        _expect(low, name, (m, rank), (torch.float32,))
    return tuple(t for t in (out, low) if t is not None)


def w4a16_lora_matmul_workspace_size(m: int, k: int, n: int, group_size: int, x_dtype: torch.dtype = torch.bfloat16,
                                     sz_dtype: torch.dtype = torch.float16,
                                     y_dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace that w4a16_lora_matmul needs for this shape (0: none)."""
    return int(load().w4a16_lora_matmul_workspace_size(m, k, n, group_size, _dtype_code(x_dtype), _dtype_code(sz_dtype),
                                                       _dtype_code(y_dtype)))


def _lora_workspace(name: str, x, m, k, n, group_size, scales, y, *more):
    """The workspace that a product asks for, from torch, beside x: (tensor that keeps it, pointer, bytes)."""
    nbytes = _workspace_bytes(name, m, k, n, group_size, _DT[x.dtype], _DT[scales.dtype], _DT[y.dtype], *more)
    if not nbytes:
        return None, None, 0
    ws = x.new_empty((nbytes,), dtype=torch.uint8)
    return ws, ws.data_ptr(), nbytes


def w4a16_lora_matmul(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                      group_size: int, a: torch.Tensor, b: torch.Tensor, scaling: torch.Tensor,
                      offsets: torch.Tensor, adapters: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
                      out: Optional[torch.Tensor] = None, u: Optional[torch.Tensor] = None):
    """y [M, N] = x . dequant(W)^T + u . B^T with u = scaling x . A^T of each row's adapter.

    a [L, R, K] and b [L, N, R] (both bf16 or both fp32, R a multiple of 8 up
    to 256), scaling float32 [L]; offsets int32 [S + 1], rising, and adapters
    int32 [S] on the GPU (never read on the host): rows offsets[s] ..
    offsets[s+1]-1 have adapter adapters[s], none if that is no number of 0 .. L-1.
    u: a float32 [M, R] tensor that takes u (rows of no adapter are left as they
    were).  out_dtype defaults to x's dtype.  The workspace comes from torch."""
    m, k, n = _int4_product(x, "x", packed, scales, zeros, group_size, False)
    count, rank, s = _check_lora(a, b, scaling, offsets, adapters, k, n)
    given = () if out is None and u is None else _given(out, (m, n), u, "u", m, rank)
    dev = _device(x, packed, scales, zeros, a, b, scaling, offsets, adapters, *given)
    y = _y_out(out, out_dtype or x.dtype, (m, n), x)
    if u is None:
        u = x.new_empty((m, rank), dtype=torch.float32)
    ws, ws_ptr, ws_bytes = _lora_workspace("w4a16_lora_matmul_workspace_size", x, m, k, n, group_size, scales, y)
    _launch(dev, load().w4a16_lora_matmul, x.data_ptr(), _DT[x.dtype], m, k, packed.data_ptr(), scales.data_ptr(),
            zeros.data_ptr(), _DT[scales.dtype], n, group_size, a.data_ptr(), b.data_ptr(), _DT[a.dtype], count, rank,
            scaling.data_ptr(), offsets.data_ptr(), adapters.data_ptr(), s, u.data_ptr(), y.data_ptr(), _DT[y.dtype],
            ws_ptr, ws_bytes)
    return y


def w4a16_matmul_t_workspace_size(m: int, k: int, n: int, group_size: int, dy_dtype: torch.dtype = torch.bfloat16,
                                  sz_dtype: torch.dtype = torch.float16,
                                  dx_dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace that w4a16_matmul_t needs for this shape (0: none)."""
    return int(load().w4a16_matmul_t_workspace_size(m, k, n, group_size, _dtype_code(dy_dtype), _dtype_code(sz_dtype),
                                                    _dtype_code(dx_dtype)))


def w4a16_matmul_t(dy: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor, group_size: int,
                   out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None):
    """dx [M, K] = dy [M, N] . dequant(W): the gradient of w4a16_matmul with respect to x.

    dy bf16 or fp32; out_dtype defaults to dy's dtype.  The workspace comes from torch."""
    m, k, n = _int4_product(dy, "dy", packed, scales, zeros, group_size, True)
    dev = _device(dy, packed, scales, zeros) if out is None else _device(dy, packed, scales, zeros, out)
    dx = _y_out(out, out_dtype or dy.dtype, (m, k), dy)
    ws, ws_ptr, ws_bytes = _lora_workspace("w4a16_matmul_t_workspace_size", dy, m, k, n, group_size, scales, dx)
    _launch(dev, load().w4a16_matmul_t, dy.data_ptr(), _DT[dy.dtype], m, k, packed.data_ptr(), scales.data_ptr(),
            zeros.data_ptr(), _DT[scales.dtype], n, group_size, dx.data_ptr(), _DT[dx.dtype], ws_ptr, ws_bytes)
    return dx


def w4a16_lora_matmul_t_workspace_size(m: int, k: int, n: int, group_size: int, rank: int, segments: int,
                                       dy_dtype: torch.dtype = torch.bfloat16, sz_dtype: torch.dtype = torch.float16,
                                       dx_dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace that w4a16_lora_matmul_t needs for this shape (0: none)."""
    return int(load().w4a16_lora_matmul_t_workspace_size(m, k, n, group_size, _dtype_code(dy_dtype),
                                                         _dtype_code(sz_dtype), _dtype_code(dx_dtype), rank, segments))


def w4a16_lora_matmul_t(dy: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                        group_size: int, a: torch.Tensor, b: torch.Tensor, scaling: torch.Tensor,
                        offsets: torch.Tensor, adapters: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
                        out: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None):
    """dx [M, K] = dy . dequant(W) + v . A with v = scaling dy . B of each row's
    adapter: the gradient of w4a16_lora_matmul with respect to x.

    Arguments as there; v: a float32 [M, R] tensor that takes v (rows of no
    adapter are left as they were).  out_dtype defaults to dy's dtype."""
    m, k, n = _int4_product(dy, "dy", packed, scales, zeros, group_size, True)
    count, rank, s = _check_lora(a, b, scaling, offsets, adapters, k, n)
    given = () if out is None and v is None else _given(out, (m, k), v, "v", m, rank)
    dev = _device(dy, packed, scales, zeros, a, b, scaling, offsets, adapters, *given)
    dx = _y_out(out, out_dtype or dy.dtype, (m, k), dy)
    if v is None:
        v = dy.new_empty((m, rank), dtype=torch.float32)
    ws, ws_ptr, ws_bytes = _lora_workspace("w4a16_lora_matmul_t_workspace_size", dy, m, k, n, group_size, scales, dx,
                                           rank, s)
    _launch(dev, load().w4a16_lora_matmul_t, dy.data_ptr(), _DT[dy.dtype], m, k, packed.data_ptr(), scales.data_ptr(),
            zeros.data_ptr(), _DT[scales.dtype], n, group_size, a.data_ptr(), b.data_ptr(), _DT[a.dtype], count, rank,
            scaling.data_ptr(), offsets.data_ptr(), adapters.data_ptr(), s, v.data_ptr(), dx.data_ptr(), _DT[dx.dtype],
            ws_ptr, ws_bytes)
    return dx


def lora_grads_workspace_size(m: int, k: int, n: int, adapters: int, rank: int,
                              dy_dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace that lora_grads needs for this shape (0: none)."""
    return int(load().lora_grads_workspace_size(m, k, n, _dtype_code(dy_dtype), adapters, rank))


def lora_grads(xq: torch.Tensor, xs: torch.Tensor, dy: torch.Tensor, u: torch.Tensor, v: torch.Tensor,
               offsets: torch.Tensor, adapters: torch.Tensor, num_adapters: int,
               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """(da [L, R, K], db [L, N, R]), float32: the gradients of num_adapters = L adapters.

    xq, xs: x's checkpoint from quantize_checkpoint_int8; dy [M, N] bf16 or
    fp32; u and v from w4a16_lora_matmul and w4a16_lora_matmul_t.  An adapter
    without rows gets zeros; rows of no adapter are not read."""
    m, k = _check_checkpoint(xq, xs)
    n = _matrix(dy, "dy")[1]
    _expect(dy, "dy", (m, n), Y_DTYPES)
    rank = _matrix(u, "u")[1]
    _expect(u, "u", (m, rank), (torch.float32,))
    _expect(v, "v", (m, rank), (torch.float32,))
    s = _check_segments(offsets, adapters)
    if num_adapters < 0:
        raise ValueError(f"num_adapters = {num_adapters} < 0")
    shapes = (num_adapters, rank, k), (num_adapters, n, rank)
    if out is not None:
        da, db = out
        _expect(da, "da", shapes[0], (torch.float32,))
        _expect(db, "db", shapes[1], (torch.float32,))
        dev = _device(xq, xs, dy, u, v, offsets, adapters, da, db)
    else:
        dev = _device(xq, xs, dy, u, v, offsets, adapters)
        da, db = u.new_empty(shapes[0]), u.new_empty(shapes[1])
    nbytes = _workspace_bytes("lora_grads_workspace_size", m, k, n, _DT[dy.dtype], num_adapters, rank)
    ws = u.new_empty((nbytes,), dtype=torch.uint8) if nbytes else None
    _launch(dev, load().lora_grads, _ptr(xq), _ptr(xs), m, k, _ptr(dy), _dtype_code(dy.dtype), n, _ptr(u), _ptr(v),
            _ptr(offsets), _ptr(adapters), s, num_adapters, rank, _ptr(da), _ptr(db),
            None if ws is None else _ptr(ws), nbytes)
    return da, db


def version() -> str:
    return load().w4_version().decode()
