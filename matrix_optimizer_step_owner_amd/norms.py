"""Layer norm and its gradients, the weight's and the bias's straight into the
packed fp32 gradient that ``adamw_tail`` takes.

Argument checks and marshalling only (C ABI in ``include/mfsdp.h``); calls run
on torch's current stream of their tensors' device, wait for nothing, can be
captured into a graph and record no autograd graph.

Source of the setting: arxivlens page, Abstract (tensors that are not whole 2D
matrices, norm gains among them, are packed for AdamW).
"""

from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _lib
from .grads import _DTYPES, _FLOATS, _call, _check, _contiguous, _gpu, _rows, _scratch, _span


def _vector(t: torch.Tensor, name: str, device, dtypes, d: int) -> int:
    _check(t, name, device, dtypes, 1)
    _contiguous(t, name, (d,))
    return t.data_ptr()


def layer_norm(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
               eps: float = 1e-5, centered: bool = True,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``(x - mean) / sqrt(variance + eps) * weight + bias`` of each row, in fp32
    and rounded once; not ``centered`` it divides by the root mean square
    (mfsdp_layer_norm).  The sum of a row's squares has to be an fp32 number.

    x: (rows, d) bf16 or fp32, rows contiguous at any stride; weight, bias: (d,)
    of one dtype, fp32 (segments of a packed tail) or bf16."""
    device = _gpu(x, "x")
    _check(x, "x", device, _FLOATS, 2)
    rows, d = x.shape
    w = _vector(weight, "weight", device, _FLOATS, d)
    b = None if bias is None else _vector(bias, "bias", device, (weight.dtype,), d)
    if out is None:
        out = x.new_empty((rows, d))
        ldo = d
    else:
        _check(out, "out", device, (x.dtype,), 2)
        ldo = _rows(out, "out", (rows, d))
    _call(device, "mfsdp_layer_norm", x.data_ptr(), _rows(x, "x"), w, b, _DTYPES[weight.dtype],
          rows, d, _DTYPES[x.dtype], centered, eps, out.data_ptr(), ldo)
    return out


@functools.lru_cache(maxsize=256)
def _grad_bytes(rows: int, d: int, dtype: int, with_bias: bool) -> int:
    need = ctypes.c_size_t(0)
    _lib.check(_lib.load().mfsdp_layer_norm_grad_workspace_size(rows, d, dtype, with_bias,
                                                                ctypes.byref(need)))
    return need.value


def layer_norm_grad(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                    dweight: torch.Tensor, dbias: Optional[torch.Tensor] = None, *,
                    eps: float = 1e-5, centered: bool = True, beta: float = 0.0,
                    out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradients of ``layer_norm`` (mfsdp_layer_norm_grad): returns dx (or writes
    ``out``), and in place
    ``dweight = beta * dweight + sum over rows of dy * (x - mean) / sqrt(variance + eps)``
    and ``dbias = beta * dbias + sum over rows of dy`` (None: not wanted).

    dy: (rows, d) in x's dtype; dweight, dbias: (d,) fp32, for example segments
    of the packed gradient of ``adamw_tail``; beta = 1 adds a micro-batch.  The
    rest as in ``layer_norm``; nothing of the forward is needed but x.

    workspace: scratch of at least mfsdp_layer_norm_grad_workspace_size bytes,
    256-byte aligned; without it one is kept per stream and host thread."""
    device = _gpu(x, "x")
    _check(x, "x", device, _FLOATS, 2)
    rows, d = x.shape
    _check(dy, "dy", device, (x.dtype,), 2)
    ldy = _rows(dy, "dy", (rows, d))
    w = _vector(weight, "weight", device, _FLOATS, d)
    f32 = (torch.float32,)
    dw = _vector(dweight, "dweight", device, f32, d)
    db = None if dbias is None else _vector(dbias, "dbias", device, f32, d)
    if out is None:
        out = x.new_empty((rows, d))
        ldo = d
    else:
        _check(out, "out", device, (x.dtype,), 2)
        ldo = _rows(out, "out", (rows, d))
    dtype = _DTYPES[x.dtype]
    need = _grad_bytes(rows, d, dtype, db is not None)
    ws = None if need == 0 and workspace is None else _scratch(device, need, workspace)
    _call(device, "mfsdp_layer_norm_grad", dy.data_ptr(), ldy, x.data_ptr(), _rows(x, "x"), w,
          _DTYPES[weight.dtype], rows, d, dtype, centered, eps, beta, out.data_ptr(), ldo, dw, db,
          *_span(ws))
    return out
