"""Binding of the training-step operators of include/precond.h: the RMS norm
with an 8-bit output and its gradients, the 8-bit form, the product of two 8-bit
matrices and the distillation loss.

As for the rest of the binding, torch tensors go where the C ABI takes device
pointers, outputs are the caller's, and the checks of sizes, alignment and
overlap are the library's.  An 8-bit matrix is a pair (q, scale) from
``empty8``: float8_e4m3fn values with rows a multiple of 16 bytes apart, and
float8_e8m0fnu scales in the library's order (``scales8`` puts them in the
matrix's).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import BF16, F32, _check, _stream, load

E4M3 = 2
BLOCK_ROW, BLOCK_TILE = 0, 1

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}
_fn = None


class _Functions:
    """The library's entry points with their argument types, looked up once."""

    def __init__(self):
        L = load()
        vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
        self.norm = L.precond_rms_norm
        self.norm.argtypes = [vp, vp, vp, vp, i32, i32, i64, i64, i64, i64, f32, vp, i64, vp, i64, vp, i64, vp, vp, vp]
        self.grad = L.precond_rms_norm_grad
        self.grad.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i64, i64, i64, i64, i64, vp, i64, vp, vp, i64, vp]
        self.grad_workspace = L.precond_rms_norm_grad_workspace
        self.grad_workspace.argtypes = [i64, i64]
        self.grad_workspace.restype = i64
        self.quantize = L.precond_quantize8
        self.quantize.argtypes = [vp, vp, i32, i64, i64, i64, vp, i32, vp, i64, vp, vp, i64, vp, vp]
        self.gemm = L.precond_gemm8
        self.gemm.argtypes = [vp, i64, i64, i64, vp, i64, vp, vp, i64, vp, vp, i64, i32, i32, vp]
        self.gemm_status = L.precond_gemm8_status
        self.gemm_status.argtypes = [vp, vp]
        self.distill = L.precond_distill
        self.distill.argtypes = [vp, vp, i32, i64, i64, i64, vp, i32, i64, vp, i32, i64, i32, vp, f32, vp, vp, i64, vp]
        for f in (self.norm, self.grad, self.quantize, self.gemm, self.gemm_status, self.distill):
            f.restype = i32


def _lib() -> _Functions:
    global _fn
    if _fn is None:
        _fn = _Functions()
    return _fn


def _dtype(t: torch.Tensor, what: str) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise TypeError(f"{what} must be float32 or bfloat16, got {t.dtype}")
    return d


def _matrix(t: torch.Tensor, what: str, shape=None, dtype=None) -> Tuple[int, int]:
    """(pointer, row pitch) of a 2-D tensor with consecutive columns."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{what} must be 2-D with consecutive columns")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    rows, cols = t.shape
    return t.data_ptr(), t.stride(0) if rows > 1 else max(t.stride(0), cols)


def _vector(t: torch.Tensor, what: str, n: int, dtype=torch.float32) -> int:
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous vector of {n}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    return t.data_ptr()


def scale_shape(rows: int, cols: int) -> Tuple[int, int, int, int, int]:
    """Shape of the scales of a rows x cols matrix in 8-bit form: [512-column group][128-row block]
    [row % 32][row // 32 % 4][block of 128 columns in the group]."""
    return (-(-cols // 512), -(-rows // 128), 32, 4, 4)


def _form8(q: torch.Tensor, scale: torch.Tensor, what: str, shape=None) -> Tuple[int, int, int]:
    """(pointer, pitch, scales' pointer) of a matrix in 8-bit form."""
    if q.dtype != torch.float8_e4m3fn:
        raise TypeError(f"{what} must be float8_e4m3fn, got {q.dtype}")
    if scale is None or scale.dtype not in (torch.float8_e8m0fnu, torch.uint8):
        raise TypeError(f"{what} needs float8_e8m0fnu (or uint8) scales")
    p, ld = _matrix(q, what, shape)
    rows, cols = q.shape
    if rows == 1:                            # a pitch that no row needs
        ld = max(ld, -(-cols // 16) * 16)
        ld = -(-ld // 16) * 16
    if not scale.is_contiguous() or scale.numel() != -(-cols // 512) * -(-rows // 128) * 512:
        raise ValueError(f"{what}'s scales must be contiguous, of shape {scale_shape(rows, cols)}")
    return p, ld, scale.data_ptr()


def empty8(rows: int, cols: int, device="cuda") -> Tuple[torch.Tensor, torch.Tensor]:
    """An uninitialised matrix in 8-bit form: (q, scale)."""
    q = torch.empty((rows, -(-cols // 16) * 16), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)[:, :cols]
    return q, torch.empty(scale_shape(rows, cols), dtype=torch.uint8, device=device).view(torch.float8_e8m0fnu)


def scales8(scale: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """The scales as a float32 matrix, rows x blocks of 128 columns."""
    g, r = scale.shape[:2]
    s = scale.view(torch.uint8).permute(1, 3, 2, 0, 4).reshape(r * 128, g * 4)[:rows, :-(-cols // 128)]
    return s.contiguous().view(torch.float8_e8m0fnu).float()


def dequantize8(q: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    """The float32 values of a matrix in 8-bit form (torch operations, for inspection and tests)."""
    rows, cols = q.shape
    return q.float() * scales8(scale, rows, cols).repeat_interleave(128, dim=1)[:, :cols]


def precond_rms_norm(h, x, weight, eps: float, residual=None, total=None, y=None, q=None, scale=None, rstd=None,
                     stream=None, raw: bool = False) -> int:
    """total = x + residual; y, and its 8-bit form (q, scale) = total / rms(total) * weight; rstd for the
    gradients.  Outputs that are None are not written."""
    f = _fn or _lib()
    dt = _dtype(x, "x")
    shape = x.shape
    px, ldx = _matrix(x, "x")
    rows, cols = shape
    pr = ldr = pt = ldt = py = ldy = pq = ldq = ps = pn = 0
    if residual is not None:
        pr, ldr = _matrix(residual, "residual", shape, x.dtype)
    if total is not None:
        pt, ldt = _matrix(total, "total", shape, x.dtype)
    if y is not None:
        py, ldy = _matrix(y, "y", shape, x.dtype)
    if q is not None:
        pq, ldq, ps = _form8(q, scale, "q", shape)
    if rstd is not None:
        pn = _vector(rstd, "rstd", rows)
    code = f.norm(h, px, pr, _vector(weight, "weight", cols, None), dt, _dtype(weight, "weight"), rows, cols, ldx, ldr, eps,
                  pt, ldt, py, ldy, pq, ldq, ps, pn, _stream(stream))
    return code if raw else _check(code, "precond_rms_norm")


def precond_rms_norm_grad_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace of precond_rms_norm_grad."""
    return _lib().grad_workspace(rows, cols)


def precond_rms_norm_grad(h, dy, x, weight, rstd, dx, dw, dresidual=None, workspace=None, stream=None,
                          raw: bool = False) -> int:
    """dx and dw of precond_rms_norm; x is the forward pass's total.  Without a workspace one comes from torch's
    allocator (on the current stream; pass your own with another ``stream``)."""
    f = _fn or _lib()
    dt = _dtype(dy, "dy")
    shape = dy.shape
    pdy, lddy = _matrix(dy, "dy")
    rows, cols = shape
    px, ldx = _matrix(x, "x", shape, dy.dtype)
    pdx, lddx = _matrix(dx, "dx", shape, dy.dtype)
    pr = ldr = 0
    if dresidual is not None:
        pr, ldr = _matrix(dresidual, "dresidual", shape, dy.dtype)
    if workspace is None:
        need = f.grad_workspace(rows, cols)
        if stream is not None and _stream(stream) != _stream(None):
            raise ValueError("give a workspace with a stream other than torch's current one")
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dy.device)
    code = f.grad(h, pdy, px, _vector(weight, "weight", cols, None), _vector(rstd, "rstd", rows), pr, dt,
                  _dtype(weight, "weight"), rows, cols, lddy, ldx, ldr, pdx, lddx, _vector(dw, "dw", cols),
                  workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream))
    return code if raw else _check(code, "precond_rms_norm_grad")


def precond_quantize8(h, x, q=None, scale=None, qt=None, scale_t=None, block: int = BLOCK_ROW,
                      x_scale: Optional[torch.Tensor] = None, stream=None, raw: bool = False) -> int:
    """The 8-bit form of x (float32, bfloat16, or itself in 8-bit form with ``x_scale``): by rows into
    (q, scale) and transposed into (qt, scale_t); either may be left out."""
    f = _fn or _lib()
    rows, cols = x.shape
    pxs = pq = ldq = ps = pqt = ldqt = pst = 0
    if x.dtype == torch.float8_e4m3fn:
        dt = E4M3
        px, ldx, pxs = _form8(x, x_scale, "x")
    else:
        dt = _dtype(x, "x")
        px, ldx = _matrix(x, "x")
        if x_scale is not None:
            raise ValueError("x_scale goes with a float8_e4m3fn x")
    if q is not None:
        pq, ldq, ps = _form8(q, scale, "q", x.shape)
    if qt is not None:
        pqt, ldqt, pst = _form8(qt, scale_t, "qt", (cols, rows))
    code = f.quantize(h, px, dt, rows, cols, ldx, pxs, block, pq, ldq, ps, pqt, ldqt, pst, _stream(stream))
    return code if raw else _check(code, "precond_quantize8")


def precond_gemm8(h, a, scale_a, b, scale_b, out, accumulate: bool = False, stream=None, raw: bool = False) -> int:
    """out = a b^T (or out += a b^T) of matrices in 8-bit form, M x K and N x K; out is float32 or bfloat16."""
    f = _fn or _lib()
    m, k = a.shape
    n = b.shape[0]
    pa, lda, psa = _form8(a, scale_a, "a")
    pb, ldb, psb = _form8(b, scale_b, "b", (n, k))
    pc, ldc = _matrix(out, "out", (m, n))
    code = f.gemm(h, m, n, k, pa, lda, psa, pb, ldb, psb, pc, ldc, _dtype(out, "out"), int(accumulate), _stream(stream))
    return code if raw else _check(code, "precond_gemm8")


def precond_gemm8_status(h, stream=None, raw: bool = False) -> int:
    """Synchronises; ECUDA if a wait inside a product's kernel ran out since the last call."""
    code = _lib().gemm_status(h, _stream(stream))
    return code if raw else _check(code, "precond_gemm8_status")


def precond_distill(h, logits, ids, teacher, loss, weight=None, temperature: float = 1.0, dlogits=None, stream=None,
                    raw: bool = False) -> int:
    """loss of every row against the teacher's top logits (``teacher`` at the vocabulary places ``ids``) and,
    with ``dlogits``, its gradient (in place if it is ``logits``)."""
    f = _fn or _lib()
    pz, ldz = _matrix(logits, "logits")
    rows, vocab = logits.shape
    top = ids.shape[1] if ids.dim() == 2 else -1
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    pi, ldi = _matrix(ids, "ids", (rows, top))
    pt, ldt = _matrix(teacher, "teacher", (rows, top))
    pw = pd = ldd = 0
    if weight is not None:
        pw = _vector(weight, "weight", rows)
    if dlogits is not None:
        pd, ldd = _matrix(dlogits, "dlogits", logits.shape, logits.dtype)
    code = f.distill(h, pz, _dtype(logits, "logits"), rows, vocab, ldz, pi, 32 if ids.dtype == torch.int32 else 64, ldi, pt,
                     _dtype(teacher, "teacher"), ldt, top, pw, temperature, _vector(loss, "loss", rows), pd, ldd,
                     _stream(stream))
    return code if raw else _check(code, "precond_distill")
