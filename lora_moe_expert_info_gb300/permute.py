"""Tokens sorted by expert and back, with their gradients.

  moe_permute             rows sorted by expert, their places, the experts' first rows
  moe_sort_pairs          the places and first rows alone
  moe_permute_backward    the gradient of the copied tokens
  moe_unpermute           rows weighted and summed back per token
  moe_unpermute_backward  the gradients of rows and weights
  MoePermute, MoeUnpermute  the same as torch.autograd functions

A pair p = t*K + k is token t's k-th choice; pairs are sorted by expert id,
stable in p.  A pair whose id is not in [0, num_experts) -- -1 to mask it -- comes
last with a zero row, and pair_pos holds ~row for it.  Tensors are bf16 or
float32; sums run in increasing k in float32, so results are bit-identical
between runs.  Every step runs in the library's kernels; nothing here
synchronises unless check=True.  All tensors are on the current CUDA device.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _check_device, _check_host, _launch_stream, _on_stream, _req, library

__all__ = ["moe_permute", "moe_sort_pairs", "moe_permute_backward", "moe_unpermute", "moe_unpermute_backward",
           "MoePermute", "MoeUnpermute"]

DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_typed = None


def _lib():
    global _typed
    if _typed is None:
        lib = library()
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        for f in (lib.moe_permute_workspace_bytes, lib.moe_sort_pairs_workspace_bytes):
            f.restype = sz
            f.argtypes = [i32] * 3
        lib.moe_permute.restype = ctypes.c_int
        lib.moe_permute.argtypes = [vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp, vp]
        lib.moe_unpermute.restype = ctypes.c_int
        lib.moe_unpermute.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp]
        lib.moe_unpermute_backward.restype = ctypes.c_int
        lib.moe_unpermute_backward.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp]
        _typed = lib
    return _typed


def _address(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _float(t: torch.Tensor, name: str, dev, ndim: int = 2) -> int:
    """Checks a contiguous bf16 or float32 tensor; its type number."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in DTYPES:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    _req(t, name, t.dtype, dev)
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    return DTYPES[t.dtype]


def _out(t: Optional[torch.Tensor], name: str, shape, dtype, dev) -> torch.Tensor:
    """A caller's output buffer, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _req(t, name, dtype, dev)
    if t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    return t


def _sort(x, topk_ids, num_experts, rows, pair_pos, expert_offsets, workspace, check, fn):
    lib = _lib()
    if not isinstance(topk_ids, torch.Tensor):
        raise TypeError("topk_ids must be a torch.Tensor")
    dev = topk_ids.device
    _req(topk_ids, "topk_ids", torch.int32, dev)
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be [num_tokens, topk]")
    T, K = topk_ids.shape
    E = int(num_experts)
    dtype = H = 0
    if x is not None:
        dtype = _float(x, "x", dev)
        H = x.shape[1]
        if x.shape[0] != T:
            raise ValueError(f"{fn}: inconsistent shapes")
    on = _launch_stream(topk_ids, fn)
    if x is not None:
        rows = _out(rows, "rows", (T * K, H), x.dtype, dev)
    # an empty tensor has no address: rows of no columns are only sorted
    copy = H > 0
    wsb = (lib.moe_permute_workspace_bytes if copy else lib.moe_sort_pairs_workspace_bytes)(T, K, E)
    if wsb == 0:
        raise ValueError(f"{fn}: unsupported sizes")
    pair_pos = _out(pair_pos, "pair_pos", (T, K), torch.int32, dev)
    expert_offsets = _out(expert_offsets, "expert_offsets", (E + 1,), torch.int32, dev)
    if workspace is not None:
        _req(workspace, "workspace", getattr(workspace, "dtype", None), dev)  # of any type
    elif wsb > 1:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev) if check else None
    code = lib.moe_permute(x.data_ptr() if copy else None, topk_ids.data_ptr(), T, K, H, E, dtype,
                           rows.data_ptr() if copy else None, pair_pos.data_ptr(), expert_offsets.data_ptr(),
                           _address(workspace), 0 if workspace is None else workspace.nbytes, _address(status), on)
    _check_host(code, fn)
    if check:
        _check_device(status, fn)
    return rows, pair_pos, expert_offsets


@_on_stream
def moe_permute(x, topk_ids, num_experts: int, rows: Optional[torch.Tensor] = None,
                pair_pos: Optional[torch.Tensor] = None, expert_offsets: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None,
                check: bool = True) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Tokens x [T, H] copied into rows sorted by expert.  Returns (rows [T*K, H],
    pair_pos int32 [T, K], expert_offsets int32 [num_experts + 1]); given buffers
    are written in place.  With check=True the stream is synchronised and ids
    other than -1 outside [0, num_experts) raise."""
    if x is None:
        raise TypeError("x must be a torch.Tensor")
    return _sort(x, topk_ids, num_experts, rows, pair_pos, expert_offsets, workspace, check, "moe_permute")


@_on_stream
def moe_sort_pairs(topk_ids, num_experts: int, pair_pos: Optional[torch.Tensor] = None,
                   expert_offsets: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None, check: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
    """The order alone: (pair_pos, expert_offsets) of moe_permute."""
    return _sort(None, topk_ids, num_experts, None, pair_pos, expert_offsets, workspace, check, "moe_sort_pairs")[1:]


def _gather(rows, pair_pos, weights, y, check, fn, rows_name):
    lib = _lib()
    if not isinstance(pair_pos, torch.Tensor):
        raise TypeError("pair_pos must be a torch.Tensor")
    dev = pair_pos.device
    _req(pair_pos, "pair_pos", torch.int32, dev)
    if pair_pos.dim() != 2:
        raise ValueError("pair_pos must be [num_tokens, topk]")
    dtype = _float(rows, rows_name, dev)
    T, K = pair_pos.shape
    H = rows.shape[1]
    if weights is not None:
        _req(weights, "topk_weights", torch.float32, dev)
    if rows.shape[0] != T * K or (weights is not None and weights.shape != (T, K)):
        raise ValueError(f"{fn}: inconsistent shapes")
    on = _launch_stream(pair_pos, fn)
    y = _out(y, "y", (T, H), rows.dtype, dev)
    if T == 0 or H == 0:
        return y
    status = torch.zeros(1, dtype=torch.int32, device=dev) if check else None
    code = lib.moe_unpermute(rows.data_ptr(), pair_pos.data_ptr(), _address(weights), T, K, H, dtype, y.data_ptr(),
                             _address(status), on)
    _check_host(code, fn)
    if check:
        _check_device(status, fn)
    return y


@_on_stream
def moe_permute_backward(d_rows, pair_pos, dx: Optional[torch.Tensor] = None, stream=None,
                         check: bool = False) -> torch.Tensor:
    """The gradient of moe_permute's x: dx[t] = sum over k of d_rows[pair_pos[t, k]]."""
    return _gather(d_rows, pair_pos, None, dx, check, "moe_permute_backward", "d_rows")


@_on_stream
def moe_unpermute(rows, pair_pos, topk_weights, y: Optional[torch.Tensor] = None, stream=None,
                  check: bool = False) -> torch.Tensor:
    """y[t] = sum over k of topk_weights[t, k] * rows[pair_pos[t, k]], masked pairs skipped."""
    if topk_weights is None:
        raise TypeError("topk_weights must be a torch.Tensor")
    return _gather(rows, pair_pos, topk_weights, y, check, "moe_unpermute", "rows")


@_on_stream
def moe_unpermute_backward(dy, rows, pair_pos, topk_weights, d_rows: Optional[torch.Tensor] = None,
                           d_weights: Optional[torch.Tensor] = None, stream=None,
                           check: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gradients of moe_unpermute: (d_rows [T*K, H], d_weights float32 [T, K]),
    zeros for masked pairs."""
    lib = _lib()
    if not isinstance(pair_pos, torch.Tensor):
        raise TypeError("pair_pos must be a torch.Tensor")
    dev = pair_pos.device
    _req(pair_pos, "pair_pos", torch.int32, dev)
    if pair_pos.dim() != 2:
        raise ValueError("pair_pos must be [num_tokens, topk]")
    dtype = _float(rows, "rows", dev)
    _req(dy, "dy", rows.dtype, dev)
    _req(topk_weights, "topk_weights", torch.float32, dev)
    T, K = pair_pos.shape
    H = rows.shape[1]
    if rows.shape[0] != T * K or dy.shape != (T, H) or topk_weights.shape != (T, K):
        raise ValueError("moe_unpermute_backward: inconsistent shapes")
    on = _launch_stream(pair_pos, "moe_unpermute_backward")
    d_rows = _out(d_rows, "d_rows", (T * K, H), rows.dtype, dev)
    d_weights = _out(d_weights, "d_weights", (T, K), torch.float32, dev)
    if T == 0 or H == 0:
        return d_rows, d_weights.zero_()
    status = torch.zeros(1, dtype=torch.int32, device=dev) if check else None
    code = lib.moe_unpermute_backward(dy.data_ptr(), rows.data_ptr(), pair_pos.data_ptr(), topk_weights.data_ptr(), T,
                                      K, H, dtype, d_rows.data_ptr(), d_weights.data_ptr(), _address(status), on)
    _check_host(code, "moe_unpermute_backward")
    if check:
        _check_device(status, "moe_unpermute_backward")
    return d_rows, d_weights


class MoePermute(torch.autograd.Function):
    """rows, pair_pos, expert_offsets = MoePermute.apply(x, topk_ids, num_experts)"""

    @staticmethod
    def forward(ctx, x, topk_ids, num_experts):
        rows, pair_pos, expert_offsets = moe_permute(x, topk_ids, num_experts, check=False)
        ctx.save_for_backward(pair_pos)
        ctx.mark_non_differentiable(pair_pos, expert_offsets)
        return rows, pair_pos, expert_offsets

    @staticmethod
    @once_differentiable
    def backward(ctx, d_rows, *_):
        return moe_permute_backward(d_rows.contiguous(), *ctx.saved_tensors), None, None


class MoeUnpermute(torch.autograd.Function):
    """y = MoeUnpermute.apply(rows, pair_pos, topk_weights)"""

    @staticmethod
    def forward(ctx, rows, pair_pos, topk_weights):
        ctx.save_for_backward(rows, pair_pos, topk_weights)
        return moe_unpermute(rows, pair_pos, topk_weights)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        d_rows, d_weights = moe_unpermute_backward(dy.contiguous(), *ctx.saved_tensors)
        return d_rows, None, d_weights
