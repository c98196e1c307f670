"""Which tokens go to which experts: the choice and its gradient, the plan that
sorts rows by expert for ``grouped_linear``, the balance bias, and the exchange
of rows between tokens' and experts' order with its gradients.

Argument checks and marshalling only (C ABI in ``include/mfsdp.h``); every call
runs on torch's current stream of its tensors' device, waits for nothing and
can be captured into a graph, and none records an autograd graph: gradients are
calls of their own.

    experts, weights = route(logits, 8, scores="sigmoid", bias=bias)
    plan = route_plan(experts, n_experts)
    xs = route_dispatch(x, plan.place)                       # rows by expert
    h = grouped_linear(xs, w, plan.offsets)
    y = route_combine(h, plan.place, weights)
    # backward
    dh, dweights = route_combine_grad(dy, h, plan.place, weights)
    dxs = grouped_linear_dgrad(dh, w, plan.offsets)
    dx = route_combine(dxs, plan.place)
    dlogits = route_grad(dweights, logits, experts, scores="sigmoid")
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib
from .grads import _DTYPES, _FLOATS, _call, _check, _contiguous, _gpu, _rows, _scratch, _span

_I32, _F32 = (torch.int32,), (torch.float32,)


class RoutePlan(NamedTuple):
    """Rows of a routing: ``offsets`` (experts + 1,) of each expert's rows, and
    ``place`` (tokens, k), the row of each choice or -1."""
    offsets: torch.Tensor
    place: torch.Tensor


def _score(scores: str) -> int:
    try:
        return _lib.ROUTE_SCORES[scores]
    except (KeyError, TypeError):
        raise ValueError(f"scores must be 'softmax' or 'sigmoid', not {scores!r}") from None


def _whole(t: torch.Tensor, name: str, device, dtypes, shape) -> int:
    """Address of a contiguous tensor of this shape."""
    _check(t, name, device, dtypes, len(shape))
    _contiguous(t, name, shape)
    return t.data_ptr()


def route(logits: torch.Tensor, k: int, *, scores: str = "softmax",
          bias: Optional[torch.Tensor] = None, groups: int = 1, top_groups: int = 1,
          renormalize: bool = True, scale: float = 1.0, mask: Optional[torch.Tensor] = None,
          experts: Optional[torch.Tensor] = None,
          weights: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The k experts of each token, int32 (tokens, k), and their weights, fp32
    (mfsdp_route).

    With s the softmax or sigmoid of a row of logits, an expert's key is s +
    bias.  Of ``groups`` groups of neighbouring experts the ``top_groups`` with
    the largest sums of their two largest keys stay; the k largest keys among
    them are chosen in descending order, ties to the lowest index, as in exact
    arithmetic.  A weight is scale * s / (sum of the chosen s + 1e-20), without
    ``renormalize`` scale * s: the bias chooses and does not weigh.

    logits: (tokens, experts) bf16 or fp32, rows contiguous at any stride; bias:
    (experts,) fp32; mask: (tokens,) bool, False for padding, whose experts are
    -1 and weights 0."""
    device = _gpu(logits, "logits")
    _check(logits, "logits", device, _FLOATS, 2)
    tokens, n = logits.shape
    ld = _rows(logits, "logits")
    b = None if bias is None else _whole(bias, "bias", device, _F32, (n,))
    m = None if mask is None else _whole(mask, "mask", device, (torch.bool,), (tokens,))
    held = min(max(k, 0), n)    # a k outside is refused below, without room for it
    if experts is None:
        experts = logits.new_empty((tokens, held), dtype=torch.int32)
    else:
        _whole(experts, "experts", device, _I32, (tokens, k))
    if weights is None:
        weights = logits.new_empty((tokens, held), dtype=torch.float32)
    else:
        _whole(weights, "weights", device, _F32, (tokens, k))
    _call(device, "mfsdp_route", logits.data_ptr(), ld, b, m, tokens, n, k, _DTYPES[logits.dtype],
          _score(scores), groups, top_groups, renormalize, scale, experts.data_ptr(),
          weights.data_ptr())
    return experts, weights


def route_grad(dweights: torch.Tensor, logits: torch.Tensor, experts: torch.Tensor, *,
               scores: str = "softmax", renormalize: bool = True, scale: float = 1.0,
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of ``route``'s logits from that of its weights, in the logits'
    dtype (mfsdp_route_grad).  dweights: (tokens, k) fp32; logits, experts,
    scores, renormalize and scale as there.  Tokens without an expert get zeros.
    The choice itself, and with it the bias, has no gradient."""
    device = _gpu(logits, "logits")
    _check(logits, "logits", device, _FLOATS, 2)
    tokens, n = logits.shape
    _check(experts, "experts", device, _I32, 2)
    k = experts.shape[1]
    _contiguous(experts, "experts", (tokens, k))
    dw = _whole(dweights, "dweights", device, _F32, (tokens, k))
    if out is None:
        out = logits.new_empty((tokens, n))
        ldo = n
    else:
        _check(out, "out", device, (logits.dtype,), 2)
        ldo = _rows(out, "out", (tokens, n))
    _call(device, "mfsdp_route_grad", dw, logits.data_ptr(), _rows(logits, "logits"),
          experts.data_ptr(), tokens, n, k, _DTYPES[logits.dtype], _score(scores), renormalize,
          scale, out.data_ptr(), ldo)
    return out


@functools.lru_cache(maxsize=256)
def _plan_bytes(tokens: int, k: int, n_experts: int) -> int:
    need = ctypes.c_size_t(0)
    _lib.check(_lib.load().mfsdp_route_plan_workspace_size(tokens, k, n_experts, ctypes.byref(need)))
    return need.value


def route_plan(experts: torch.Tensor, n_experts: int, *, offsets: Optional[torch.Tensor] = None,
               place: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> RoutePlan:
    """Rows of the choices, sorted by expert, tokens in order within one
    (mfsdp_route_plan).  experts: (tokens, k) int32; a number outside [0,
    n_experts) is no choice and gets place -1.  The plan's rows are the first
    offsets[-1] of tokens * k.

    workspace: scratch of at least mfsdp_route_plan_workspace_size bytes,
    256-byte aligned; without it one is kept per stream and host thread."""
    device = _gpu(experts, "experts")
    _check(experts, "experts", device, _I32, 2)
    _contiguous(experts, "experts")
    tokens, k = experts.shape
    need = _plan_bytes(tokens, k, n_experts)    # refuses sizes before there is room for them
    if offsets is None:
        offsets = experts.new_empty((n_experts + 1,))
    else:
        _whole(offsets, "offsets", device, _I32, (n_experts + 1,))
    if place is None:
        place = experts.new_empty((tokens, k))
    else:
        _whole(place, "place", device, _I32, (tokens, k))
    ws = None if need == 0 and workspace is None else _scratch(device, need, workspace)
    _call(device, "mfsdp_route_plan", experts.data_ptr(), tokens, k, n_experts, offsets.data_ptr(),
          place.data_ptr(), *_span(ws))
    return RoutePlan(offsets, place)


def route_balance(bias: torch.Tensor, counts: torch.Tensor, rate: float) -> torch.Tensor:
    """Moves the balance bias, in place: up by ``rate`` for an expert with fewer
    choices than the mean, down for one with more (mfsdp_route_balance).  bias:
    (experts,) fp32; counts: (experts,) int32 or int64, for example
    ``plan.offsets.diff()`` summed over the ranks.  Returns bias."""
    device = _gpu(bias, "bias")
    _check(bias, "bias", device, _F32, 1)
    _contiguous(bias, "bias")
    c = _whole(counts, "counts", device, (torch.int32, torch.int64), bias.shape)
    _call(device, "mfsdp_route_balance", bias.data_ptr(), c, counts.element_size(), bias.numel(),
          rate)
    return bias


def _place(place: torch.Tensor, device) -> Tuple[int, int]:
    _check(place, "place", device, _I32, 2)
    _contiguous(place, "place")
    return place.shape


def route_dispatch(x: torch.Tensor, place: torch.Tensor,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Tokens' rows in their experts' order: ``out[place[t, j]] = x[t]``
    (mfsdp_route_dispatch).

    x: (tokens, d) bf16 or fp32, rows contiguous at any stride; place: (tokens,
    k) int32, a row outside ``out`` is none.  ``out`` has tokens * k rows unless
    it is given; rows of no choice are left as they are in it (and undefined in
    one made here), and a row that two choices name gets either's values.  Its gradient is ``route_combine`` without weights."""
    device = _gpu(x, "x")
    _check(x, "x", device, _FLOATS, 2)
    tokens, d = x.shape
    t, k = _place(place, device)
    if t != tokens:
        raise ValueError(f"place has {t} tokens, expected {tokens}")
    if out is None:
        out = x.new_empty((tokens * k, d))
        ldo = d
    else:
        _check(out, "out", device, (x.dtype,), 2)
        ldo = _rows(out, "out", (out.shape[0], d))
    _call(device, "mfsdp_route_dispatch", x.data_ptr(), _rows(x, "x"), place.data_ptr(), tokens, k,
          out.shape[0], d, _DTYPES[x.dtype], out.data_ptr(), ldo)
    return out


def route_combine(h: torch.Tensor, place: torch.Tensor, weights: Optional[torch.Tensor] = None, *,
                  beta: float = 0.0, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Experts' rows back to their tokens:
    ``out[t] = beta * out[t] + sum over j of weights[t, j] * h[place[t, j]]``,
    in fp32 and rounded once (mfsdp_route_combine).

    h: (rows, d) bf16 or fp32, rows contiguous at any stride; place: (tokens, k)
    int32, a row outside h is none; weights: (tokens, k) fp32, None for ones
    (the gradient of ``route_dispatch``).  beta != 0 needs ``out``, for example
    with a shared expert's rows, and adds to it."""
    device = _gpu(h, "h")
    _check(h, "h", device, _FLOATS, 2)
    rows, d = h.shape
    tokens, k = _place(place, device)
    w = None if weights is None else _whole(weights, "weights", device, _F32, (tokens, k))
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs an out to add to")
        out = h.new_empty((tokens, d))
        ldo = d
    else:
        _check(out, "out", device, (h.dtype,), 2)
        ldo = _rows(out, "out", (tokens, d))
    _call(device, "mfsdp_route_combine", h.data_ptr(), _rows(h, "h"), place.data_ptr(), w, tokens,
          k, rows, d, _DTYPES[h.dtype], beta, out.data_ptr(), ldo)
    return out


def route_combine_grad(dy: torch.Tensor, h: torch.Tensor, place: torch.Tensor,
                       weights: torch.Tensor, *, dh: Optional[torch.Tensor] = None,
                       dweights: Optional[torch.Tensor] = None
                       ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Gradients of ``route_combine``: ``dh[place[t, j]] = weights[t, j] * dy[t]``
    and ``dweights[t, j] = <dy[t], h[place[t, j]]>`` (0 for no choice;
    mfsdp_route_combine_grad).  dy: (tokens, d) in h's dtype; dh: like h, rows of
    no choice left as they are (undefined in one made here); dweights: (tokens,
    k) fp32."""
    device = _gpu(h, "h")
    _check(h, "h", device, _FLOATS, 2)
    rows, d = h.shape
    tokens, k = _place(place, device)
    _check(dy, "dy", device, (h.dtype,), 2)
    ldy = _rows(dy, "dy", (tokens, d))
    w = _whole(weights, "weights", device, _F32, (tokens, k))
    if dh is None:
        dh = h.new_empty((rows, d))
        ldo = d
    else:
        _check(dh, "dh", device, (h.dtype,), 2)
        ldo = _rows(dh, "dh", (rows, d))
    if dweights is None:
        dweights = weights.new_empty((tokens, k))
    else:
        _whole(dweights, "dweights", device, _F32, (tokens, k))
    _call(device, "mfsdp_route_combine_grad", dy.data_ptr(), ldy, h.data_ptr(), _rows(h, "h"),
          place.data_ptr(), w, tokens, k, rows, d, _DTYPES[h.dtype], dh.data_ptr(), ldo,
          dweights.data_ptr())
    return dh, dweights
