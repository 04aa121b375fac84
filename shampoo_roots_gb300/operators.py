"""Binding of the training-step operators of include/precond.h: the RMS norm and
the layer norm with an 8-bit output and their gradients, the 8-bit form, the product
of two 8-bit matrices, the distillation and the policy loss, and the norm and
clipping of a list of gradients.

As for the rest of the binding, torch tensors go where the C ABI takes device
pointers, outputs are the caller's, and the checks of sizes, alignment and
overlap are the library's.  An 8-bit matrix is a pair (q, scale) from
``empty8``: float8_e4m3fn values with rows a multiple of 16 bytes apart, and
float8_e8m0fnu scales in the library's order (``scales8`` puts them in the
matrix's).  A ``stream`` of None is torch's current stream on the device of the
tensors.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional, Tuple

import torch

from . import BF16, F32, HERE, OK, _check, _stream, load

BLOCK_ROW, BLOCK_TILE = 0, 1
E4M3 = 2
BINDING_PATH = os.path.join(HERE, "_binding.so")


def _load_binding():
    """csrc/binding.c with the library's entry points; raises if it has not been built."""
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is missing: build it with shampoo_roots_gb300.build.build()")
    spec = importlib.util.spec_from_file_location("shampoo_roots_gb300._binding", BINDING_PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    L = load()
    L.precond_rms_norm_grad_workspace.argtypes = [ctypes.c_int64, ctypes.c_int64]
    L.precond_rms_norm_grad_workspace.restype = ctypes.c_int64
    L.precond_layer_norm_grad_workspace.argtypes = [ctypes.c_int64, ctypes.c_int64]
    L.precond_layer_norm_grad_workspace.restype = ctypes.c_int64
    L.precond_gemm8_status.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    L.precond_gemm8_status.restype = ctypes.c_int
    m.set_up((torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.uint8, torch.int32, torch.int64),
             torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else _current_stream,
             tuple(ctypes.cast(f, ctypes.c_void_p).value for f in (
                 L.precond_rms_norm, L.precond_rms_norm_grad, L.precond_rms_norm_grad_workspace, L.precond_quantize8, L.precond_gemm8,
                 L.precond_distill, L.precond_distill_workspace, L.precond_layer_norm, L.precond_layer_norm_grad,
                 L.precond_layer_norm_grad_workspace, L.precond_policy, L.precond_list_create, L.precond_list_destroy,
                 L.precond_list_workspace, L.precond_grad_norm, L.precond_clip_grads)), _allocator())
    return m


def _allocator():
    """(allocate, delete, current device) of torch's caching allocator, what torch.cuda.caching_allocator_alloc calls;
    None where this torch has them under other names."""
    names = ("_cuda_cudaCachingAllocator_raw_alloc", "_cuda_cudaCachingAllocator_raw_delete", "_cuda_getDevice")
    found = tuple(getattr(torch._C, n, None) for n in names)
    return None if None in found else found


def _current_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


_b = _load_binding()


def scale_shape(rows: int, cols: int) -> Tuple[int, int, int, int, int]:
    """Shape of the scales of a rows x cols matrix in 8-bit form: [512-column group][128-row block]
    [row % 32][row // 32 % 4][block of 128 columns in the group]."""
    return (-(-cols // 512), -(-rows // 128), 32, 4, 4)


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
    code = _b.rms_norm(h, x, weight, eps, residual, total, y, q, scale, rstd, stream)
    return code if raw or code == OK else _check(code, "precond_rms_norm")


def precond_rms_norm_grad_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace of precond_rms_norm_grad."""
    return load().precond_rms_norm_grad_workspace(rows, cols)


def precond_rms_norm_grad(h, dy, x, weight, rstd, dx, dw, dresidual=None, workspace=None, stream=None,
                          raw: bool = False) -> int:
    """dx and dw of precond_rms_norm; x is the forward pass's total.  Without a workspace one comes from torch's
    allocator (on the current stream; give one together with another ``stream``)."""
    code = _b.rms_norm_grad(h, dy, x, weight, rstd, dx, dw, dresidual, workspace, stream)
    return code if raw or code == OK else _check(code, "precond_rms_norm_grad")


def precond_quantize8(h, x, q=None, scale=None, qt=None, scale_t=None, block: int = BLOCK_ROW,
                      x_scale: Optional[torch.Tensor] = None, stream=None, raw: bool = False) -> int:
    """The 8-bit form of x (float32, bfloat16, or itself in 8-bit form with ``x_scale``): by rows into
    (q, scale) and transposed into (qt, scale_t); either may be left out."""
    code = _b.quantize8(h, x, q, scale, qt, scale_t, block, x_scale, stream)
    return code if raw or code == OK else _check(code, "precond_quantize8")


def precond_gemm8(h, a, scale_a, b, scale_b, out, accumulate: bool = False, stream=None, raw: bool = False) -> int:
    """out = a b^T (or out += a b^T) of matrices in 8-bit form, M x K and N x K; out is float32 or bfloat16."""
    code = _b.gemm8(h, a, scale_a, b, scale_b, out, accumulate, stream)
    return code if raw or code == OK else _check(code, "precond_gemm8")


def precond_gemm8_status(h, stream=None, raw: bool = False) -> int:
    """Synchronises; ECUDA if a wait inside a product's kernel ran out since the last call."""
    code = load().precond_gemm8_status(h, _stream(stream))
    return code if raw or code == OK else _check(code, "precond_gemm8_status")


def precond_distill_workspace(rows: int, vocab: int, top: int, dtype: torch.dtype, in_place: bool = False) -> int:
    """Bytes of workspace of precond_distill for logits of float32 or bfloat16."""
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"logits must be float32 or bfloat16, got {dtype}")
    L = load()
    L.precond_distill_workspace.restype = ctypes.c_int64
    L.precond_distill_workspace.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    return L.precond_distill_workspace(rows, vocab, top, F32 if dtype == torch.float32 else BF16, int(in_place))


def precond_distill(h, logits, ids, teacher, loss, weight=None, temperature: float = 1.0, dlogits=None, workspace=None,
                    stream=None, raw: bool = False) -> int:
    """loss of every row against the teacher's top logits (``teacher`` at the vocabulary places ``ids``) and,
    with ``dlogits``, its gradient (in place if it is ``logits``).  Without a workspace one comes from torch's
    allocator where the call needs it (on the current stream; give one together with another ``stream``).
    ``temperature`` is 1e-18 to 1e18."""
    code = _b.distill(h, logits, ids, teacher, loss, weight, temperature, dlogits, workspace, stream)
    return code if raw or code == OK else _check(code, "precond_distill")


def precond_layer_norm(h, x, weight, eps: float, bias=None, residual=None, total=None, y=None, q=None, scale=None, mean=None,
                       rstd=None, stream=None, raw: bool = False) -> int:
    """total = x + residual; y, and its 8-bit form (q, scale) = (total - mean) * rstd * weight + bias; mean and rstd
    for the gradients.  Outputs that are None are not written."""
    code = _b.layer_norm(h, x, weight, eps, bias, residual, total, y, q, scale, mean, rstd, stream)
    return code if raw or code == OK else _check(code, "precond_layer_norm")


def precond_layer_norm_grad_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace of precond_layer_norm_grad."""
    return load().precond_layer_norm_grad_workspace(rows, cols)


def precond_layer_norm_grad(h, dy, x, weight, mean, rstd, dx, dw, db=None, dresidual=None, workspace=None, stream=None,
                            raw: bool = False) -> int:
    """dx, dw and db of precond_layer_norm; x is the forward pass's total.  The workspace as in
    precond_rms_norm_grad."""
    code = _b.layer_norm_grad(h, dy, x, weight, mean, rstd, dx, dw, db, dresidual, workspace, stream)
    return code if raw or code == OK else _check(code, "precond_layer_norm_grad")


def precond_policy(h, logits, ids, advantage=None, old_logp=None, ref_logp=None, weight=None, temperature: float = 1.0,
                   clip_low: float = 0.2, clip_high: float = 0.2, kl: float = 0.0, loss=None, logp=None, dlogits=None,
                   stream=None, raw: bool = False) -> int:
    """The clipped policy loss of every row's taken token ``ids``, its log probability and, with ``dlogits``, the
    gradient (in place if it is ``logits``).  Without ``advantage`` the log probabilities alone.  ``old_logp`` None is
    a ratio of 1; ``kl`` weighs the KL term against ``ref_logp``.  Rows of weight 0 and ids outside the vocabulary are
    left out: zero loss, logp and gradient.

    A preference loss over pairs of sequences takes two calls: one for logp, whose sums per sequence give each row its
    coefficient, and one with those as ``-advantage`` for the gradient."""
    code = _b.policy(h, logits, ids, advantage, old_logp, ref_logp, weight, temperature, clip_low, clip_high, kl, loss, logp,
                     dlogits, stream)
    return code if raw or code == OK else _check(code, "precond_policy")


class TensorList:
    """Tensors (float32 or bfloat16, dense, apart from one another) that precond_grad_norm and precond_clip_grads
    take together.  It keeps them alive; make it once for buffers that stay."""

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        code, self._list, self.workspace = _b.tensor_list(self.tensors)    # workspace: bytes, of a call
        _check(code, "precond_list_create")

    def __len__(self) -> int:
        return len(self.tensors)


def _listed(grads) -> TensorList:
    return grads if isinstance(grads, TensorList) else TensorList(grads)


def precond_grad_norm(h, grads, norm, workspace=None, stream=None, raw: bool = False) -> int:
    """norm (one float32 on the device) = the 2-norm of all elements of ``grads``, a TensorList or a sequence of
    tensors.  The workspace as in precond_rms_norm_grad."""
    g = _listed(grads)
    code = _b.grad_norm(h, g._list, g.tensors[0] if g.tensors else None, norm, workspace, stream)
    return code if raw or code == OK else _check(code, "precond_grad_norm")


def precond_clip_grads(h, grads, max_norm: float, norm, given: bool = False, workspace=None, stream=None,
                       raw: bool = False) -> int:
    """``grads`` *= max_norm / norm in place where norm > max_norm.  The norm is computed and left in ``norm``, or, with
    ``given``, read there.  Gradients whose norm is not finite stay as they are."""
    g = _listed(grads)
    code = _b.clip_grads(h, g._list, g.tensors[0] if g.tensors else None, max_norm, norm, given, workspace, stream)
    return code if raw or code == OK else _check(code, "precond_clip_grads")
