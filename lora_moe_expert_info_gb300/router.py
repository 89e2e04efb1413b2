"""The router's choice of experts, the balance loss, and their gradients.

  moe_route           topk_ids and topk_weights from the router's logits
  moe_balance_loss    the loss that keeps experts evenly used, and the tokens per expert
  moe_route_backward  the gradient of the logits from the weights, the loss or both
  MoeRoute            all of it as a torch.autograd function

The ids and weights are those that the expert layers, permute and fp4 take; an id
of -1 masks a pair.  Logits are bf16 or float32, [T, E]; one that is not finite
counts as -inf and its expert is never chosen (NaN and +inf are reported by
check=True).  Choice scores are compared in 64 bits where 32 do not tell them apart,
ties go to the lowest index, and sums run in a fixed order: results are bit-identical
between runs.  Sigmoids are float32: logits below -87 may weigh nothing.  Every step
runs in the library's kernels; nothing here synchronises unless check=True.  All
tensors are contiguous and on the current CUDA device.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _check_device, _check_host, _launch_stream, _on_stream, _req, library
from .permute import _address, _float, _out

__all__ = ["moe_route", "moe_balance_loss", "moe_route_backward", "MoeRoute", "SCORING"]

SCORING = {"softmax": 0, "sigmoid": 1}
_typed = None


def _lib():
    global _typed
    if _typed is None:
        lib = library()
        vp, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
        lib.moe_route.restype = ctypes.c_int
        lib.moe_route.argtypes = [vp] * 3 + [i32] * 8 + [f32] + [vp] * 4
        lib.moe_balance_loss_workspace_bytes.restype = sz
        lib.moe_balance_loss_workspace_bytes.argtypes = [i32] * 2
        lib.moe_balance_loss.restype = ctypes.c_int
        lib.moe_balance_loss.argtypes = [vp] * 3 + [i32] * 5 + [vp] * 3 + [sz] + [vp] * 2
        lib.moe_route_backward.restype = ctypes.c_int
        lib.moe_route_backward.argtypes = [vp] * 6 + [i32] * 6 + [f32] + [vp] * 3
        _typed = lib
    return _typed


def _scoring(scoring: str) -> int:
    if scoring not in SCORING:
        raise ValueError(f"scoring must be one of {sorted(SCORING)}, got {scoring!r}")
    return SCORING[scoring]


def _logits(logits):
    """Checks logits [T, E]; (type number, T, E, device)."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    dtype = _float(logits, "logits", logits.device)
    if logits.shape[1] == 0:
        raise ValueError("logits have no experts")
    return dtype, *logits.shape, logits.device


def _mask(token_mask, T: int, dev):
    if token_mask is not None:
        _req(token_mask, "token_mask", torch.bool, dev)
        if token_mask.shape != (T,):
            raise ValueError(f"token_mask must have shape ({T},)")


def _ids(topk_ids, T: int, dev) -> int:
    """Checks topk_ids [T, K]; K."""
    _req(topk_ids, "topk_ids", torch.int32, dev)
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T or topk_ids.shape[1] == 0:
        raise ValueError("topk_ids must be [num_tokens, topk]")
    return topk_ids.shape[1]


@_on_stream
def moe_route(logits, topk: int, scoring: str = "softmax", bias: Optional[torch.Tensor] = None, num_groups: int = 1,
              topk_groups: int = 1, renormalize: bool = True, scale: float = 1.0,
              token_mask: Optional[torch.Tensor] = None, topk_ids: Optional[torch.Tensor] = None,
              topk_weights: Optional[torch.Tensor] = None, stream=None,
              check: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """(topk_ids int32, topk_weights float32), both [T, topk], the best expert first.

    scoring "softmax" chooses by the logits, "sigmoid" by sigmoid(logits) + bias (a
    float32 [E] that only the choice sees).  With num_groups > 1 the experts of the
    topk_groups best groups stand to choice: a group's score is its best expert's
    (softmax) or the sum of its two best (sigmoid).  Weights are the chosen experts'
    softmax or sigmoid, divided by their sum (renormalize), times scale.  Tokens
    whose token_mask (bool [T]) is False, and places that no expert is left for, get
    id -1 and weight 0."""
    code = _scoring(scoring)
    dtype, T, E, dev = _logits(logits)
    K = int(topk)
    if K < 1:
        raise ValueError("topk must be positive")
    if bias is not None:
        if not code:
            raise ValueError("moe_route: a bias goes with sigmoid scoring")
        _req(bias, "bias", torch.float32, dev)
        if bias.shape != (E,):
            raise ValueError(f"bias must have shape ({E},)")
    _mask(token_mask, T, dev)
    on = _launch_stream(logits, "moe_route")
    topk_ids = _out(topk_ids, "topk_ids", (T, K), torch.int32, dev)
    topk_weights = _out(topk_weights, "topk_weights", (T, K), torch.float32, dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev) if check else None
    _check_host(_lib().moe_route(logits.data_ptr(), _address(bias), _address(token_mask), T, E, K, num_groups,
                                 topk_groups, dtype, code, bool(renormalize), scale, topk_ids.data_ptr(),
                                 topk_weights.data_ptr(), _address(status), on), "moe_route")
    if check:
        _check_device(status, "moe_route")
    return topk_ids, topk_weights


@_on_stream
def moe_balance_loss(logits, topk_ids, scoring: str = "softmax", token_mask: Optional[torch.Tensor] = None,
                     loss: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None,
                     check: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """(loss, counts): loss = E / (K N^2) sum_e c_e sum_t p_te, a float32 scalar that is
    1 for evenly used experts, with N the tokens that are not masked, c_e their pairs
    of expert e, and p = softmax(logits) or sigmoid(logits) over its sum; counts int32
    [E + 1]: c, then N."""
    lib = _lib()
    code = _scoring(scoring)
    dtype, T, E, dev = _logits(logits)
    K = _ids(topk_ids, T, dev)
    _mask(token_mask, T, dev)
    on = _launch_stream(logits, "moe_balance_loss")
    loss = _out(loss, "loss", (), torch.float32, dev)
    counts = _out(counts, "counts", (E + 1,), torch.int32, dev)
    if workspace is not None:
        _req(workspace, "workspace", getattr(workspace, "dtype", None), dev)  # of any type
    else:
        wsb = lib.moe_balance_loss_workspace_bytes(T, E)
        if wsb > 1:
            workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev) if check else None
    _check_host(lib.moe_balance_loss(logits.data_ptr(), topk_ids.data_ptr(), _address(token_mask), T, E, K, dtype,
                                     code, loss.data_ptr(), counts.data_ptr(), _address(workspace),
                                     0 if workspace is None else workspace.nbytes, _address(status), on),
                "moe_balance_loss")
    if check:
        _check_device(status, "moe_balance_loss")
    return loss, counts


@_on_stream
def moe_route_backward(logits, topk_ids, d_weights: Optional[torch.Tensor] = None,
                       counts: Optional[torch.Tensor] = None, d_loss: Optional[torch.Tensor] = None,
                       scoring: str = "softmax", renormalize: bool = True, scale: float = 1.0,
                       token_mask: Optional[torch.Tensor] = None, d_logits: Optional[torch.Tensor] = None, stream=None,
                       check: bool = False) -> torch.Tensor:
    """d_logits [T, E] in the logits' type, from d_weights float32 [T, K] (the gradient
    of moe_route's weights), from d_loss (one float32 on the device, with the counts of
    moe_balance_loss), or from both in one pass; the other arguments as they were given
    to those."""
    code = _scoring(scoring)
    dtype, T, E, dev = _logits(logits)
    K = _ids(topk_ids, T, dev)
    if d_weights is None and d_loss is None:
        raise ValueError("moe_route_backward: neither d_weights nor d_loss")
    if (counts is None) != (d_loss is None):
        raise ValueError("moe_route_backward: counts and d_loss go together")
    if d_weights is not None:
        _req(d_weights, "d_weights", torch.float32, dev)
        if d_weights.shape != (T, K):
            raise ValueError("moe_route_backward: inconsistent shapes")
    if counts is not None:
        _req(counts, "counts", torch.int32, dev)
        _req(d_loss, "d_loss", torch.float32, dev)
        if counts.shape != (E + 1,) or d_loss.numel() != 1:
            raise ValueError("moe_route_backward: inconsistent shapes")
    _mask(token_mask, T, dev)
    on = _launch_stream(logits, "moe_route_backward")
    d_logits = _out(d_logits, "d_logits", (T, E), logits.dtype, dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev) if check else None
    _check_host(_lib().moe_route_backward(logits.data_ptr(), topk_ids.data_ptr(), _address(d_weights), _address(counts),
                                          _address(d_loss), _address(token_mask), T, E, K, dtype, code,
                                          bool(renormalize), scale, d_logits.data_ptr(), _address(status), on),
                "moe_route_backward")
    if check:
        _check_device(status, "moe_route_backward")
    return d_logits


class MoeRoute(torch.autograd.Function):
    """topk_weights, topk_ids, loss, counts = MoeRoute.apply(logits, topk, scoring, bias,
    num_groups, topk_groups, renormalize, scale, token_mask): moe_route and
    moe_balance_loss with one gradient of the logits (topk_weights and loss are
    differentiable).  Arguments from scoring on may be left out."""

    @staticmethod
    def forward(ctx, logits, topk, scoring="softmax", bias=None, num_groups=1, topk_groups=1, renormalize=True,
                scale=1.0, token_mask=None):
        ids, weights = moe_route(logits, topk, scoring, bias, num_groups, topk_groups, renormalize, scale, token_mask)
        loss, counts = moe_balance_loss(logits, ids, scoring, token_mask)
        ctx.save_for_backward(logits, ids, counts, token_mask)
        ctx.how = scoring, renormalize, scale
        ctx.mark_non_differentiable(ids, counts)
        ctx.set_materialize_grads(False)
        return weights, ids, loss, counts

    @staticmethod
    @once_differentiable
    def backward(ctx, d_weights, _ids, d_loss, _counts):
        none = (None,) * 8
        if d_weights is None and d_loss is None:
            return None, *none
        logits, ids, counts, token_mask = ctx.saved_tensors
        d = moe_route_backward(logits, ids, None if d_weights is None else d_weights.contiguous(),
                               None if d_loss is None else counts, d_loss, *ctx.how, token_mask)
        return d, *none
