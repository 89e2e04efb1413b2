"""The residual's addition and the root-mean-square norm before the experts.

  rms_norm           y and the new residual stream
  rms_norm_fp8       the same, with y in 8 bits as the W8A8 layer takes its activations
  fp8_dequantize     those 8 bits back to numbers
  rms_norm_backward  the gradients
  RmsNorm            rms_norm as a torch.autograd function

Per row r = x + residual, rounded to the tensors' type (r = x without a residual),
and y = r * weight / sqrt(mean(r^2) + eps).  Rows are bf16 or float32, the weight
either of them.  Sums are held in float32 in a fixed order, so results are
bit-identical between runs.  Every step runs in the library's kernels; nothing here
synchronises.  All tensors are contiguous and on the current CUDA device.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch
from torch.autograd.function import once_differentiable

from . import _check_host, _launch_stream, _on_stream, _req, library
from .permute import DTYPES, _address, _float, _out

__all__ = ["rms_norm", "rms_norm_fp8", "fp8_dequantize", "rms_norm_backward", "RmsNorm"]

GROUP = 128  # columns of an 8-bit scale
_typed = None


def _lib():
    global _typed
    if _typed is None:
        lib = library()
        vp, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
        lib.moe_rms_norm.restype = ctypes.c_int
        lib.moe_rms_norm.argtypes = [vp] * 3 + [i32] * 4 + [f32] + [vp] * 5
        lib.moe_fp8_dequantize.restype = ctypes.c_int
        lib.moe_fp8_dequantize.argtypes = [vp] * 2 + [i32] * 3 + [vp] * 2
        lib.moe_rms_norm_backward_workspace_bytes.restype = sz
        lib.moe_rms_norm_backward_workspace_bytes.argtypes = [i32] * 3
        lib.moe_rms_norm_backward.restype = ctypes.c_int
        lib.moe_rms_norm_backward.argtypes = [vp] * 4 + [i32] * 4 + [f32] + [vp] * 3 + [sz, vp]
        _typed = lib
    return _typed


def _weight(weight, H: int, dev) -> int:
    dtype = _float(weight, "weight", dev, 1)
    if weight.shape[0] != H:
        raise ValueError(f"weight must have {H} entries")
    return dtype


def _norm(x, weight, eps, residual, y, residual_out, codes, exps, eight, with_y, fn):
    lib = _lib()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = x.device
    dtype = _float(x, "x", dev)
    T, H = x.shape
    if H == 0:
        raise ValueError("x has no columns")
    w_dtype = _weight(weight, H, dev)
    if residual is not None:
        _req(residual, "residual", x.dtype, dev)
        if residual.shape != x.shape:
            raise ValueError(f"{fn}: inconsistent shapes")
    elif residual_out is not None:
        raise ValueError(f"{fn}: residual_out without a residual")
    on = _launch_stream(x, fn)
    if with_y:
        y = _out(y, "y", (T, H), x.dtype, dev)
    r = x if residual is None else _out(residual_out, "residual_out", (T, H), x.dtype, dev)
    if eight:
        codes = _out(codes, "codes", (T, H), torch.uint8, dev)
        exps = _out(exps, "exps", (T, (H + GROUP - 1) // GROUP), torch.uint8, dev)
    _check_host(lib.moe_rms_norm(x.data_ptr(), _address(residual), weight.data_ptr(), T, H, dtype, w_dtype, eps,
                                 y.data_ptr() if with_y else None, None if residual is None else r.data_ptr(),
                                 _address(codes), _address(exps), on), fn)
    return codes, exps, y, r


@_on_stream
def rms_norm(x, weight, eps: float = 1e-6, residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(y, r) of x [T, H]: r = x + residual (x itself without one), y its norm
    times weight [H].  y may be x (which without a residual is r too, and then gone)
    and residual_out may be residual."""
    return _norm(x, weight, eps, residual, y, residual_out, None, None, False, True, "rms_norm")[2:]


@_on_stream
def rms_norm_fp8(x, weight, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
                 codes: Optional[torch.Tensor] = None, exps: Optional[torch.Tensor] = None,
                 y: Optional[torch.Tensor] = None, residual_out: Optional[torch.Tensor] = None, with_y: bool = True,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor], torch.Tensor]:
    """(codes, exps, y, r): as rms_norm, and y in 8 bits, uint8 codes [T, H] (E4M3)
    and uint8 exps [T, ceil(H / 128)] with y about code * 2^(exp - 127) per group of
    128 columns -- what fused_moe_lora_forward_fp8_w8a8 makes of y itself.
    with_y=False: y is not written (and None)."""
    if not with_y and y is not None:
        raise ValueError("rms_norm_fp8: y given, with_y=False")
    return _norm(x, weight, eps, residual, y, residual_out, codes, exps, True, with_y, "rms_norm_fp8")


@_on_stream
def fp8_dequantize(codes, exps, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The numbers of codes [T, H] and exps [T, ceil(H / 128)], in bf16 (which holds
    them exactly above 2^-126) or float32."""
    if dtype not in DTYPES:
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
    if not isinstance(codes, torch.Tensor):
        raise TypeError("codes must be a torch.Tensor")
    dev = codes.device
    _req(codes, "codes", torch.uint8, dev)
    _req(exps, "exps", torch.uint8, dev)
    if codes.dim() != 2 or exps.shape != (codes.shape[0], (codes.shape[1] + GROUP - 1) // GROUP):
        raise ValueError("fp8_dequantize: inconsistent shapes")
    on = _launch_stream(codes, "fp8_dequantize")
    out = _out(out, "out", codes.shape, dtype, dev)
    if out.numel():
        _check_host(_lib().moe_fp8_dequantize(codes.data_ptr(), exps.data_ptr(), codes.shape[0], codes.shape[1],
                                              DTYPES[dtype], out.data_ptr(), on), "fp8_dequantize")
    return out


@_on_stream
def rms_norm_backward(dy, r, weight, eps: float = 1e-6, d_r: Optional[torch.Tensor] = None,
                      dx: Optional[torch.Tensor] = None, d_weight: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(dx, d_weight float32): the gradient of x, which is also the residual's, from
    dy, the gradient of y, and d_r, what reaches r by other ways (the residual
    stream).  r as rms_norm returned it.  dx may be dy or d_r."""
    lib = _lib()
    if not isinstance(r, torch.Tensor):
        raise TypeError("r must be a torch.Tensor")
    dev = r.device
    dtype = _float(r, "r", dev)
    T, H = r.shape
    if H == 0:
        raise ValueError("r has no columns")
    w_dtype = _weight(weight, H, dev)
    for t, name in ((dy, "dy"), (d_r, "d_r")):
        if t is not None or name == "dy":
            _req(t, name, r.dtype, dev)
            if t.shape != r.shape:
                raise ValueError("rms_norm_backward: inconsistent shapes")
    on = _launch_stream(r, "rms_norm_backward")
    dx = _out(dx, "dx", (T, H), r.dtype, dev)
    d_weight = _out(d_weight, "d_weight", (H,), torch.float32, dev)
    if workspace is None:
        wsb = lib.moe_rms_norm_backward_workspace_bytes(T, H, dtype)
        workspace = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    else:
        _req(workspace, "workspace", getattr(workspace, "dtype", None), dev)  # of any type
    _check_host(lib.moe_rms_norm_backward(dy.data_ptr(), r.data_ptr(), weight.data_ptr(), _address(d_r), T, H, dtype,
                                          w_dtype, eps, dx.data_ptr(), d_weight.data_ptr(), workspace.data_ptr(),
                                          workspace.nbytes, on), "rms_norm_backward")
    return dx, d_weight


class RmsNorm(torch.autograd.Function):
    """y, r = RmsNorm.apply(x, weight, eps, residual); residual may be None (r is then x)."""

    @staticmethod
    def forward(ctx, x, weight, eps, residual):
        y, r = rms_norm(x, weight, eps, residual)
        ctx.save_for_backward(r, weight)
        ctx.eps, ctx.added = eps, residual is not None
        ctx.set_materialize_grads(False)
        return y, r

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, d_r):
        r, weight = ctx.saved_tensors
        if dy is None:
            return d_r, None, None, d_r if ctx.added else None
        dx, dw = rms_norm_backward(dy.contiguous(), r, weight, ctx.eps, None if d_r is None else d_r.contiguous())
        return dx, dw.to(weight.dtype), None, dx if ctx.added else None
