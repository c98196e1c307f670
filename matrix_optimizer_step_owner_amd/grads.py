"""The gradients that the owner-local step takes, where they are more than one
plain matrix product: experts' matrices (``grouped_linear`` and its gradients),
8-bit activation checkpoints, and the embedding table.

Argument checks and marshalling only (C ABI in ``include/mfsdp.h``); every call
runs on torch's current stream of its tensors' device, waits for nothing and
can be captured into a graph.  None of them records an autograd graph: the
gradients are calls of their own, and write where the step reads them --
``grouped_linear_wgrad`` into the stacked ``(experts, n, k)`` gradient whose
views ``grad[e]`` a ``MuonStep`` takes, ``embedding_grad`` into the table's
segment of the packed gradient of ``adamw_tail``.

Source of the setting: arxivlens page, Abstract (the owner holds whole 2D
weights with their whole gradients; the other tensors are packed for AdamW).
"""

from __future__ import annotations

import ctypes
import threading
from typing import Callable, Dict, Optional, Tuple

import torch

from . import _lib

#: columns of an activation row that share one checkpoint scale
CKPT_BLOCK = 128

_DTYPES = {torch.float32: _lib.DTYPE_F32, torch.bfloat16: _lib.DTYPE_BF16}
_FLOATS = tuple(_DTYPES)


# The current device and the handle of its current stream, without what
# torch.cuda.current_device and current_stream (a Stream object) add around
# them: together over a microsecond a call.  Looked up when called: a torch
# without a GPU backend has neither.
_C = torch._C


def _raw_stream(index: int) -> int:
    return _C._cuda_getCurrentRawStream(index)


def _check(t: torch.Tensor, name: str, device, dtypes, dim: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.ndim != dim:
        raise ValueError(f"{name} must be {dim}D")


def _contiguous(t: torch.Tensor, name: str, shape=None) -> None:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _rows(t: torch.Tensor, name: str, shape=None) -> int:
    """Row stride of a matrix whose rows are contiguous (any stride between rows)."""
    rows, cols = have = t.shape
    if shape is not None and have != shape:
        raise ValueError(f"{name} has shape {tuple(have)}, expected {tuple(shape)}")
    ld, inner = t.stride()
    if cols > 1 and inner != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:
        return max(cols, 1)
    if ld < cols:
        raise ValueError(f"rows of {name} overlap")
    return ld


def _gpu(t: torch.Tensor, name: str) -> torch.device:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


_functions: Dict[str, Callable] = {}


def _call(device: torch.device, name: str, *args) -> None:
    """The library's function on the current stream of `device`, made current."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(_lib.load(), name)
    index = device.index
    if index == _C._cuda_getDevice():
        status = fn(*args, _C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index))
    if status:
        _lib.check(status)


# The workspaces kept for calls that bring none, one per (device, stream) and
# host thread.  Calls on one stream run in order and can share one, but only if
# their launches are enqueued in order too: another thread may run between the
# launches of one call, so each has its own.
_kept = threading.local()


def _scratch(device: torch.device, nbytes: int, given: Optional[torch.Tensor]) -> torch.Tensor:
    """The caller's workspace; else this thread's kept one of the current
    stream; else, under capture, one that belongs to the graph (a kept one could
    be replayed by two graphs at once).  The caller holds it until the launches
    are enqueued."""
    if given is not None:
        if not isinstance(given, torch.Tensor):
            raise TypeError("workspace must be a tensor")
        _check(given, "workspace", device, (given.dtype,), given.dim())
        _contiguous(given, "workspace")
        return given
    with torch.cuda.device(device):
        if torch.cuda.is_current_stream_capturing():
            return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        key = (device.index, _raw_stream(device.index))
        kept = _kept.__dict__
        ws = kept.get(key)
        if ws is None or ws.numel() < nbytes:
            kept.pop(key, None)
            ws = kept[key] = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        return ws


def _grouped_args(act: torch.Tensor, name: str, weight: torch.Tensor, wname: str,
                  offsets: torch.Tensor, dtypes):
    """Device, and the shape (experts, n, k) of the stacked matrices."""
    device = _gpu(act, name)
    _check(act, name, device, _FLOATS, 2)
    _check(offsets, "offsets", device, (torch.int32,), 1)
    _check(weight, wname, device, dtypes, 3)
    _contiguous(weight, wname)
    shape = weight.shape
    _contiguous(offsets, "offsets", (shape[0] + 1,))
    return device, shape


def _grouped_rows(name: str, act: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor,
                  out: Optional[torch.Tensor], forward: bool) -> torch.Tensor:
    arg = "x" if forward else "dy"
    dtype = act.dtype if isinstance(act, torch.Tensor) else None
    device, (experts, n, k) = _grouped_args(act, arg, weight, "weight", offsets, (dtype,))
    rows = act.shape[0]
    width, to = (k, n) if forward else (n, k)
    ld = _rows(act, arg, (rows, width))
    if out is None:
        out = act.new_empty((rows, to))
        ldo = to
    else:
        _check(out, "out", device, (dtype,), 2)
        ldo = _rows(out, "out", (rows, to))
    _call(device, name, act.data_ptr(), ld, weight.data_ptr(), offsets.data_ptr(), experts, rows,
          n, k, _DTYPES[dtype], out.data_ptr(), ldo)
    return out


def grouped_linear(x: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``out[r] = x[r] @ weight[e].T`` for the rows offsets[e] <= r < offsets[e+1]
    of every expert e (mfsdp_grouped_linear).

    x: (rows, k) bf16 or fp32, rows contiguous at any stride, sorted by expert;
    weight: (experts, n, k) contiguous, x's dtype; offsets: (experts + 1,) int32
    on the GPU, non-decreasing, read there.  Rows of no expert are left as they
    are in ``out`` (and undefined in an ``out`` made here)."""
    return _grouped_rows("mfsdp_grouped_linear", x, weight, offsets, out, True)


def grouped_linear_dgrad(dy: torch.Tensor, weight: torch.Tensor, offsets: torch.Tensor,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of ``grouped_linear``'s input: ``out[r] = dy[r] @ weight[e]``
    (mfsdp_grouped_linear_dgrad).  dy: (rows, n); out: (rows, k); the rest as
    there."""
    return _grouped_rows("mfsdp_grouped_linear_dgrad", dy, weight, offsets, out, False)


def _wgrad_scratch(device: torch.device, sizes,
                   given: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    """The workspace of a weight gradient, None if it needs none."""
    need = ctypes.c_size_t(0)
    _lib.check(_lib.load().mfsdp_grouped_linear_wgrad_workspace_size(*sizes, ctypes.byref(need)))
    if need.value == 0 and given is None:
        return None
    return _scratch(device, need.value, given)


def _span(ws: Optional[torch.Tensor]):
    """(address, bytes) of a workspace."""
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def grouped_linear_wgrad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                         grad: torch.Tensor, beta: float = 0.0,
                         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradients of the experts' matrices, in place:
    ``grad[e] = beta * grad[e] + dy[rows of e].T @ x[rows of e]``
    (mfsdp_grouped_linear_wgrad).

    dy: (rows, n), x: (rows, k), one dtype; grad: (experts, n, k) contiguous in
    that dtype or fp32, each ``grad[e]`` as ``muon_step`` takes it.  beta = 1
    adds a micro-batch to what is there; beta = 0 does not read it.  An expert
    without rows gets ``beta * grad[e]``.  Returns grad.

    workspace: scratch of at least mfsdp_grouped_linear_wgrad_workspace_size
    bytes, 256-byte aligned; without it one is kept per stream and host thread.
    One that is given is for one stream and one host thread at a time."""
    dtype = dy.dtype if isinstance(dy, torch.Tensor) else None
    device, (experts, n, k) = _grouped_args(dy, "dy", grad, "grad", offsets,
                                            (dtype, torch.float32))
    rows = dy.shape[0]
    _check(x, "x", device, (dtype,), 2)
    ws = _wgrad_scratch(device, (experts, rows, n, k, _DTYPES[dtype]), workspace)
    _call(device, "mfsdp_grouped_linear_wgrad", dy.data_ptr(), _rows(dy, "dy", (rows, n)),
          x.data_ptr(), _rows(x, "x", (rows, k)), offsets.data_ptr(), experts, rows, n, k,
          _DTYPES[dtype], grad.data_ptr(), _DTYPES[grad.dtype], beta, *_span(ws))
    return grad


def _check_codes(codes: torch.Tensor, device, rows: int, k: int) -> None:
    _check(codes, "codes", device, (torch.int8,), 2)
    _contiguous(codes, "codes", (rows, k))


def _check_scales(scales: torch.Tensor, device, rows: int, k: int) -> None:
    _check(scales, "scales", device, (torch.uint8,), 2)
    _contiguous(scales, "scales", (rows, -(-k // CKPT_BLOCK)))


def grouped_linear_wgrad_ckpt(dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                              offsets: torch.Tensor, grad: torch.Tensor, beta: float = 0.0,
                              workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``grouped_linear_wgrad`` with x as its 8-bit checkpoint, (codes, scales)
    of ``ckpt_quantize`` (mfsdp_grouped_linear_wgrad_ckpt): the gradient for the
    restored x, which is never written out.  workspace: as there."""
    dtype = dy.dtype if isinstance(dy, torch.Tensor) else None
    device, (experts, n, k) = _grouped_args(dy, "dy", grad, "grad", offsets,
                                            (dtype, torch.float32))
    rows = dy.shape[0]
    _check_codes(codes, device, rows, k)
    _check_scales(scales, device, rows, k)
    ws = _wgrad_scratch(device, (experts, rows, n, k, _DTYPES[dtype]), workspace)
    _call(device, "mfsdp_grouped_linear_wgrad_ckpt", dy.data_ptr(), _rows(dy, "dy", (rows, n)),
          codes.data_ptr(), scales.data_ptr(), offsets.data_ptr(), experts, rows, n, k,
          _DTYPES[dtype], grad.data_ptr(), _DTYPES[grad.dtype], beta, *_span(ws))
    return grad


def ckpt_quantize(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                  scales: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """8-bit checkpoint of an activation (mfsdp_ckpt_quantize): int8 codes
    (rows, k) and uint8 scales (rows, ceil(k / 128)).

    Each block of 128 columns of a row is held as whole numbers q and one power
    of two 2^e (scale byte e + 127), the smallest with max|x| <= 127 * 2^e;
    x is held as q * 2^e, off by at most half of 2^e.  x: (rows, k) bf16 or
    fp32, rows contiguous at any stride."""
    device = _gpu(x, "x")
    _check(x, "x", device, _FLOATS, 2)
    rows, k = x.shape
    if codes is None:
        codes = x.new_empty((rows, k), dtype=torch.int8)
    else:
        _check_codes(codes, device, rows, k)
    if scales is None:
        scales = x.new_empty((rows, -(-k // CKPT_BLOCK)), dtype=torch.uint8)
    else:
        _check_scales(scales, device, rows, k)
    _call(device, "mfsdp_ckpt_quantize", x.data_ptr(), _rows(x, "x"), rows, k,
          _DTYPES[x.dtype], codes.data_ptr(), scales.data_ptr())
    return codes, scales


def ckpt_restore(codes: torch.Tensor, scales: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The activation that a checkpoint holds, in bf16 or fp32 (exact in both;
    mfsdp_ckpt_restore).  With ``out`` its dtype is taken."""
    device = _gpu(codes, "codes")
    _check(codes, "codes", device, (torch.int8,), 2)
    _contiguous(codes, "codes")
    rows, k = codes.shape
    _check_scales(scales, device, rows, k)
    if out is None:
        if dtype not in _DTYPES:
            raise TypeError(f"unsupported dtype {dtype}")
        out = codes.new_empty((rows, k), dtype=dtype)
    else:
        _check(out, "out", device, _FLOATS, 2)
    _call(device, "mfsdp_ckpt_restore", codes.data_ptr(), scales.data_ptr(), rows, k,
          _DTYPES[out.dtype], out.data_ptr(), _rows(out, "out", (rows, k)))
    return out


def _check_tokens(tokens: torch.Tensor, device) -> int:
    """Bytes of a token."""
    if not isinstance(tokens, torch.Tensor):
        raise TypeError("tokens must be a tensor")
    _check(tokens, "tokens", device, (torch.int64, torch.int32), tokens.ndim)
    _contiguous(tokens, "tokens")
    return 8 if tokens.dtype is torch.int64 else 4


def _embedding_out(out: torch.Tensor, dtype: Optional[torch.dtype], device, n: int,
                   d: int) -> int:
    """Row stride of the caller's output."""
    _check(out, "out", device, _FLOATS if dtype is None else (dtype,), 2)
    if out.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {out.dtype}")
    return _rows(out, "out", (n, d))


def embedding(table: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0,
              dtype: Optional[torch.dtype] = None,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``scale * table[token]`` for a list of tokens, computed in fp32 and
    rounded once (mfsdp_embedding).

    table: (vocab, d) contiguous, bf16 or fp32; tokens: int32 or int64 of any
    shape, contiguous; a token outside [0, vocab) stands for padding and gives
    a row of zeros.  Returns tokens.shape + (d,) in ``dtype`` (default the
    table's), or writes ``out``, (number of tokens, d) with rows at any
    stride."""
    device = _gpu(table, "table")
    _check(table, "table", device, _FLOATS, 2)
    _contiguous(table, "table")
    size = _check_tokens(tokens, device)
    vocab, d = table.shape
    n = tokens.numel()
    if out is None:
        dtype = table.dtype if dtype is None else dtype
        if dtype not in _DTYPES:
            raise TypeError(f"unsupported dtype {dtype}")
        out = table.new_empty((*tokens.shape, d), dtype=dtype)
        ldo = d
    else:
        ldo = _embedding_out(out, dtype, device, n, d)
        dtype = out.dtype
    _call(device, "mfsdp_embedding", table.data_ptr(), _DTYPES[table.dtype], vocab, d,
          tokens.data_ptr(), size, n, scale, out.data_ptr(), ldo, _DTYPES[dtype])
    return out


def embedding_grad(dy: torch.Tensor, tokens: torch.Tensor, grad: torch.Tensor, *,
                   scale: float = 1.0, beta: float = 0.0,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of ``embedding``'s table, in place:
    ``grad[v] = beta * grad[v] + scale * sum of dy over the tokens equal to v``
    (mfsdp_embedding_grad).

    dy: (number of tokens, d) bf16 or fp32, rows contiguous at any stride;
    grad: (vocab, d) fp32 contiguous, for example the table's segment of the
    packed gradient that ``adamw_tail`` takes.  The sums run over the tokens in
    sorted order and depend on the inputs alone.  beta = 1 adds a micro-batch
    and leaves the rows without a token untouched.  Returns grad.

    workspace: scratch of at least mfsdp_embedding_grad_workspace_size bytes,
    256-byte aligned; without it one is kept per stream and host thread.  One
    that is given is for one stream and one host thread at a time."""
    device = _gpu(dy, "dy")
    _check(dy, "dy", device, _FLOATS, 2)
    _check(grad, "grad", device, (torch.float32,), 2)
    _contiguous(grad, "grad")
    size = _check_tokens(tokens, device)
    vocab, d = grad.shape
    n = tokens.numel()
    ld = _rows(dy, "dy", (n, d))
    need = ctypes.c_size_t(0)
    _lib.check(_lib.load().mfsdp_embedding_grad_workspace_size(n, vocab, d, ctypes.byref(need)))
    ws = _scratch(device, need.value, workspace)
    _call(device, "mfsdp_embedding_grad", dy.data_ptr(), ld, _DTYPES[dy.dtype],
          tokens.data_ptr(), size, n, vocab, d, scale, beta, grad.data_ptr(), *_span(ws))
    return grad
