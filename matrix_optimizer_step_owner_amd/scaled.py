"""Products grouped by expert in 8-bit floats: e4m3 codes with one power of two
per block of 128, made from activations and matrices, and multiplied.

Argument checks and marshalling only (C ABI in ``include/mfsdp.h``); calls run
on torch's current stream of their tensors' device, wait for nothing, can be
captured into a graph and record no autograd graph.

    codes, scales, tcodes, tscales = scaled_quantize_weight(w, both=True)   # once a step
    y = scaled_linear(*scaled_quantize(x), codes, scales, offsets)
    dx = scaled_linear(*scaled_quantize(dy), tcodes, tscales, offsets)      # input gradient

The weight gradient stays ``grouped_linear_wgrad``: the step's matrices take
gradients that are not rounded to 8 bits.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from .grads import _DTYPES, _FLOATS, _call, _check, _contiguous, _gpu, _rows

#: columns of an activation row, and rows and columns of a matrix, that share one scale
SCALED_BLOCK = 128

_CODE = (torch.float8_e4m3fn,)
_BYTE = (torch.uint8,)


def _blocks(n: int) -> int:
    return -(-n // SCALED_BLOCK)


def scaled_quantize(x: torch.Tensor, codes: Optional[torch.Tensor] = None,
                    scales: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """8-bit copy of an activation (mfsdp_scaled_quantize): e4m3 codes (rows, k
    filled up with zeros to a multiple of 128) and uint8 scales (rows, ceil(k /
    128)).

    Each block of 128 columns of a row is held as code * 2^e with e = byte - 127,
    2^e the smallest power of two with max|x| <= 448 * 2^e.  x: (rows, k) bf16 or
    fp32, rows contiguous at any stride."""
    device = _gpu(x, "x")
    _check(x, "x", device, _FLOATS, 2)
    rows, k = x.shape
    nb = _blocks(k)
    if codes is None:
        codes = x.new_empty((rows, nb * SCALED_BLOCK), dtype=torch.float8_e4m3fn)
    else:
        _check(codes, "codes", device, _CODE, 2)
        _contiguous(codes, "codes", (rows, nb * SCALED_BLOCK))
    if scales is None:
        scales = x.new_empty((rows, nb), dtype=torch.uint8)
    else:
        _check(scales, "scales", device, _BYTE, 2)
        _contiguous(scales, "scales", (rows, nb))
    _call(device, "mfsdp_scaled_quantize", x.data_ptr(), _rows(x, "x"), rows, k, _DTYPES[x.dtype],
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def scaled_quantize_weight(weight: torch.Tensor, *, both: bool = False):
    """8-bit copy of stacked matrices (mfsdp_scaled_quantize_weight): e4m3 codes
    (experts, n, k filled up to a multiple of 128) and uint8 scales (experts,
    ceil(n / 128), ceil(k / 128)), one per 128 x 128 block; with ``both`` also
    the transposed copy, (experts, k, n filled up) and its scales, for the input
    gradient.  weight: (experts, n, k) contiguous, bf16 or fp32."""
    device = _gpu(weight, "weight")
    _check(weight, "weight", device, _FLOATS, 3)
    _contiguous(weight, "weight")
    experts, n, k = weight.shape
    nb, kb = _blocks(n), _blocks(k)
    out = [weight.new_empty((experts, n, kb * SCALED_BLOCK), dtype=torch.float8_e4m3fn),
           weight.new_empty((experts, nb, kb), dtype=torch.uint8)]
    if both:
        out += [weight.new_empty((experts, k, nb * SCALED_BLOCK), dtype=torch.float8_e4m3fn),
                weight.new_empty((experts, kb, nb), dtype=torch.uint8)]
    at = [t.data_ptr() for t in out] + [None] * (4 - len(out))
    _call(device, "mfsdp_scaled_quantize_weight", weight.data_ptr(), experts, n, k,
          _DTYPES[weight.dtype], *at)
    return tuple(out)


def scaled_linear(codes: torch.Tensor, scales: torch.Tensor, weight_codes: torch.Tensor,
                  weight_scales: torch.Tensor, offsets: torch.Tensor,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``grouped_linear`` of 8-bit copies: ``out[r] = x[r] @ weight[e].T`` for the
    rows offsets[e] <= r < offsets[e+1], of the values that the codes stand for
    (mfsdp_scaled_linear).  The input gradient is the same call with dy's codes
    and the transposed copy of the matrices.

    codes, scales: of ``scaled_quantize``; weight_codes, weight_scales: of
    ``scaled_quantize_weight``; offsets: (experts + 1,) int32 on the GPU.  out:
    (rows, n) bf16, rows contiguous at any stride.  Rows of no expert are left
    as they are in it (and undefined in one made here).  Sums keep 13 bits below
    the largest of eight neighbouring products, as the 8-bit matrix
    instructions do, and are fp32 beyond that."""
    device = _gpu(codes, "codes")
    _check(codes, "codes", device, _CODE, 2)
    _check(weight_codes, "weight_codes", device, _CODE, 3)
    rows, depth = codes.shape
    experts, n, wdepth = weight_codes.shape
    if depth != wdepth or depth % SCALED_BLOCK != 0:
        raise ValueError(f"codes have depth {depth}, weight_codes {wdepth}: both must be one "
                         f"multiple of {SCALED_BLOCK}")
    _contiguous(codes, "codes")
    _contiguous(weight_codes, "weight_codes")
    kb = depth // SCALED_BLOCK
    _check(scales, "scales", device, _BYTE, 2)
    _contiguous(scales, "scales", (rows, kb))
    _check(weight_scales, "weight_scales", device, _BYTE, 3)
    _contiguous(weight_scales, "weight_scales", (experts, _blocks(n), kb))
    _check(offsets, "offsets", device, (torch.int32,), 1)
    _contiguous(offsets, "offsets", (experts + 1,))
    if out is None:
        out = codes.new_empty((rows, n), dtype=torch.bfloat16)
        ldo = n
    else:
        _check(out, "out", device, (torch.bfloat16,), 2)
        ldo = _rows(out, "out", (rows, n))
    _call(device, "mfsdp_scaled_linear", codes.data_ptr(), scales.data_ptr(),
          weight_codes.data_ptr(), weight_scales.data_ptr(), offsets.data_ptr(), experts, rows, n,
          depth, out.data_ptr(), ldo)
    return out
