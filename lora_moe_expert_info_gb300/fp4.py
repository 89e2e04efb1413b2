"""Microscaled 4-bit floats: quantisation, and the experts' products on the FP4
tensor cores.

  fp4_quantize            a matrix, or a stack of matrices (weights)
  fp4_quantize_permuted   tokens, written to the sorted rows of their pairs
  fp4_quantize_swiglu     sorted rows [gate | up] to the codes of up * SiLU(gate)
  fp4_dequantize          codes and scales back to numbers
  fp4_expert_product      sorted rows times their expert's matrix
  fp4_moe_forward         the expert layer over all of these

Formats: "mxfp4" (blocks of 32 columns, power-of-two scales) and "nvfp4" (blocks
of 16, E4M3 scales under a float32 tensor scale).  Codes are uint8 [..., 16 *
ceil(cols / 32)], two per byte; scales uint8 [row blocks, atoms, 32, 4, 4] in
512-byte atoms of 128 rows by 4 blocks (see the C header).  Rows sorted by expert
come from permute.moe_sort_pairs or permute.moe_permute.  Every step runs in the
library's kernels; nothing here synchronises unless check=True.  All tensors are
on the current CUDA device.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _check_device, _check_host, _launch_stream, _on_stream, _req, library
from .permute import DTYPES, _address, _float, _out, moe_sort_pairs, moe_unpermute

__all__ = ["fp4_quantize", "fp4_quantize_permuted", "fp4_quantize_swiglu", "fp4_dequantize", "fp4_expert_product",
           "fp4_moe_forward", "FORMATS"]

FORMATS = {"mxfp4": 0, "nvfp4": 1}
_typed = None


def _lib():
    global _typed
    if _typed is None:
        lib = library()
        vp, i32 = ctypes.c_void_p, ctypes.c_int32
        lib.moe_fp4_pitch.restype = ctypes.c_int64
        lib.moe_fp4_pitch.argtypes = [i32]
        lib.moe_fp4_scale_atoms.restype = i32
        lib.moe_fp4_scale_atoms.argtypes = [i32, i32]
        for name, args in (("quantize", [vp] + [i32] * 5 + [vp] * 4),
                           ("quantize_permuted", [vp] * 4 + [i32] * 6 + [vp] * 5),
                           ("quantize_swiglu", [vp] * 2 + [i32] * 5 + [vp] * 5),
                           ("dequantize", [vp] * 3 + [i32] * 4 + [vp, i32, vp, vp]),
                           ("expert_product", [vp] * 7 + [i32] * 5 + [vp] * 3)):
            f = getattr(lib, "moe_fp4_" + name)
            f.restype = ctypes.c_int
            f.argtypes = args
        _typed = lib
    return _typed


def _format(fmt: str) -> int:
    if fmt not in FORMATS:
        raise ValueError(f"fmt must be one of {sorted(FORMATS)}, got {fmt!r}")
    return FORMATS[fmt]


def _pitch(cols: int) -> int:
    return (cols + 31) // 32 * 16


def _atoms(cols: int, fmt: int) -> int:
    per = 64 if fmt else 128
    return (cols + per - 1) // per


def _scale(t: Optional[torch.Tensor], name: str, n: int, fmt: int, dev):
    if t is None:
        return
    if not fmt:
        raise ValueError(f"{name}: mxfp4 has no tensor scale")
    _req(t, name, torch.float32, dev)
    if t.numel() != n:
        raise ValueError(f"{name} must have {n} entries")


def _offsets(t: torch.Tensor, dev) -> int:
    """Checks expert_offsets [E + 1]; E."""
    _req(t, "expert_offsets", torch.int32, dev)
    if t.dim() != 1 or t.numel() < 2:
        raise ValueError("expert_offsets must be [num_experts + 1]")
    return t.numel() - 1


def _outputs(codes, scales, rows, blocks, cols, fmt, dev):
    return (_out(codes, "codes", (*rows, _pitch(cols)), torch.uint8, dev),
            _out(scales, "scales", (*blocks, _atoms(cols, fmt), 32, 4, 4), torch.uint8, dev))


def _status(check: bool, dev):
    return torch.zeros(1, dtype=torch.int32, device=dev) if check else None


def _done(code: int, status, fn: str):
    _check_host(code, fn)
    if status is not None:
        _check_device(status, fn)


@_on_stream
def fp4_quantize(x, fmt: str = "nvfp4", tensor_scale: Optional[torch.Tensor] = None,
                 codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(codes, scales) of a matrix x [rows, cols] or of a stack [E, rows, cols],
    bf16 or float32; tensor_scale float32 [1] or [E] (nvfp4).  The scales of a
    matrix are [ceil(rows / 128), ...], those of a stack have E in front."""
    f = _format(fmt)
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() not in (2, 3):
        raise ValueError("x must be [rows, cols] or [matrices, rows, cols]")
    dev = x.device
    dtype = _float(x, "x", dev, x.dim())
    lead = x.shape[:-2]
    rows, cols = x.shape[-2:]
    n = lead[0] if lead else 1
    if cols == 0:
        raise ValueError("x has no columns")
    _scale(tensor_scale, "tensor_scale", n, f, dev)
    on = _launch_stream(x, "fp4_quantize")
    codes, scales = _outputs(codes, scales, (*lead, rows), (*lead, (rows + 127) // 128), cols, f, dev)
    if n * rows:
        _check_host(_lib().moe_fp4_quantize(x.data_ptr(), n, rows, cols, dtype, f, _address(tensor_scale),
                                            codes.data_ptr(), scales.data_ptr(), on), "fp4_quantize")
    return codes, scales


@_on_stream
def fp4_quantize_permuted(x, topk_ids, pair_pos, expert_offsets, fmt: str = "nvfp4",
                          tensor_scale: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
                          scales: Optional[torch.Tensor] = None, stream=None,
                          check: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Tokens x [T, cols] quantised once and written to the sorted rows of their
    pairs: (codes [T*K, .], scales [T*K // 128 + E, ...]).  topk_ids, pair_pos and
    expert_offsets as the sort took and left them; tensor_scale float32 [1]."""
    f = _format(fmt)
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    dev = x.device
    dtype = _float(x, "x", dev)
    _req(topk_ids, "topk_ids", torch.int32, dev)
    _req(pair_pos, "pair_pos", torch.int32, dev)
    E = _offsets(expert_offsets, dev)
    T, cols = x.shape
    if topk_ids.dim() != 2 or topk_ids.shape[0] != T or topk_ids.shape != pair_pos.shape:
        raise ValueError("fp4_quantize_permuted: inconsistent shapes")
    if cols == 0:
        raise ValueError("x has no columns")
    K = topk_ids.shape[1]
    _scale(tensor_scale, "tensor_scale", 1, f, dev)
    on = _launch_stream(x, "fp4_quantize_permuted")
    codes, scales = _outputs(codes, scales, (T * K,), (T * K // 128 + E,), cols, f, dev)
    if T:
        status = _status(check, dev)
        _done(_lib().moe_fp4_quantize_permuted(x.data_ptr(), topk_ids.data_ptr(), pair_pos.data_ptr(),
                                               expert_offsets.data_ptr(), T, K, cols, E, dtype, f,
                                               _address(tensor_scale), codes.data_ptr(), scales.data_ptr(),
                                               _address(status), on), status,
              "fp4_quantize_permuted")
    return codes, scales


@_on_stream
def fp4_quantize_swiglu(gate_up, expert_offsets, fmt: str = "nvfp4", tensor_scale: Optional[torch.Tensor] = None,
                        codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None, stream=None,
                        check: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Sorted rows gate_up [P, 2 * cols] (gate, then up) to the codes of up *
    gate / (1 + exp(-gate)): (codes [P, .], scales [P // 128 + E, ...])."""
    f = _format(fmt)
    if not isinstance(gate_up, torch.Tensor):
        raise TypeError("gate_up must be a torch.Tensor")
    dev = gate_up.device
    dtype = _float(gate_up, "gate_up", dev)
    E = _offsets(expert_offsets, dev)
    P, cols = gate_up.shape[0], gate_up.shape[1] // 2
    if gate_up.shape[1] % 2 or cols == 0:
        raise ValueError("gate_up must have an even number of columns")
    _scale(tensor_scale, "tensor_scale", 1, f, dev)
    on = _launch_stream(gate_up, "fp4_quantize_swiglu")
    codes, scales = _outputs(codes, scales, (P,), (P // 128 + E,), cols, f, dev)
    if P:
        status = _status(check, dev)
        _done(_lib().moe_fp4_quantize_swiglu(gate_up.data_ptr(), expert_offsets.data_ptr(), P, cols, E, dtype, f,
                                             _address(tensor_scale), codes.data_ptr(), scales.data_ptr(),
                                             _address(status), on), status, "fp4_quantize_swiglu")
    return codes, scales


@_on_stream
def fp4_dequantize(codes, scales, cols: int, fmt: str = "nvfp4", tensor_scale: Optional[torch.Tensor] = None,
                   expert_offsets: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The numbers of codes [rows, .] or [E, rows, .], in bf16 or float32.  With
    expert_offsets the rows are sorted by expert (their scales lie by expert, one
    tensor scale) and rows that are no expert's are zeros."""
    f = _format(fmt)
    if dtype not in DTYPES:
        raise TypeError(f"dtype must be bfloat16 or float32, got {dtype}")
    if not isinstance(codes, torch.Tensor):
        raise TypeError("codes must be a torch.Tensor")
    dev = codes.device
    _req(codes, "codes", torch.uint8, dev)
    _req(scales, "scales", torch.uint8, dev)
    cols = int(cols)
    if cols < 1 or codes.dim() not in ((2,) if expert_offsets is not None else (2, 3)):
        raise ValueError("fp4_dequantize: inconsistent shapes")
    lead, rows = codes.shape[:-2], codes.shape[-2]
    if expert_offsets is not None:
        n = _offsets(expert_offsets, dev)
        blocks = (rows // 128 + n,)
    else:
        n = lead[0] if lead else 1
        blocks = (*lead, (rows + 127) // 128)
    if codes.shape[-1] != _pitch(cols) or scales.shape != (*blocks, _atoms(cols, f), 32, 4, 4):
        raise ValueError("fp4_dequantize: inconsistent shapes")
    _scale(tensor_scale, "tensor_scale", 1 if expert_offsets is not None else n, f, dev)
    on = _launch_stream(codes, "fp4_dequantize")
    out = _out(out, "out", (*lead, rows, cols), dtype, dev)
    if out.numel():
        _check_host(_lib().moe_fp4_dequantize(codes.data_ptr(), scales.data_ptr(), _address(expert_offsets), n, rows,
                                              cols, f, _address(tensor_scale), DTYPES[dtype], out.data_ptr(), on),
                    "fp4_dequantize")
    return out


@_on_stream
def fp4_expert_product(a_codes, a_scales, expert_offsets, w_codes, w_scales, cols: int, fmt: str = "nvfp4",
                       a_tensor_scale: Optional[torch.Tensor] = None, w_tensor_scale: Optional[torch.Tensor] = None,
                       y: Optional[torch.Tensor] = None, stream=None, check: bool = True,
                       status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [P, N] bf16 of sorted rows (a_codes [P, .], scales by expert) times their
    expert's matrix (w_codes [E, N, .]), both with `cols` columns; tensor scales
    float32 [1] and [E] (nvfp4).  Rows that are no expert's (before
    expert_offsets[0], from expert_offsets[E] on) are zeros."""
    f = _format(fmt)
    if not isinstance(a_codes, torch.Tensor):
        raise TypeError("a_codes must be a torch.Tensor")
    dev = a_codes.device
    for t, n in ((a_codes, "a_codes"), (a_scales, "a_scales"), (w_codes, "w_codes"), (w_scales, "w_scales")):
        _req(t, n, torch.uint8, dev)
    E = _offsets(expert_offsets, dev)
    cols = int(cols)
    if a_codes.dim() != 2 or w_codes.dim() != 3 or cols < 1:
        raise ValueError("fp4_expert_product: inconsistent shapes")
    P, N = a_codes.shape[0], w_codes.shape[1]
    pitch, atom = _pitch(cols), (_atoms(cols, f), 32, 4, 4)
    if (a_codes.shape[1] != pitch or w_codes.shape != (E, N, pitch)
            or a_scales.shape != (P // 128 + E, *atom)
            or w_scales.shape != (E, (N + 127) // 128, *atom)):
        raise ValueError("fp4_expert_product: inconsistent shapes")
    _scale(a_tensor_scale, "a_tensor_scale", 1, f, dev)
    _scale(w_tensor_scale, "w_tensor_scale", E, f, dev)
    if status is not None:
        _req(status, "status", torch.int32, dev)
    on = _launch_stream(a_codes, "fp4_expert_product")
    y = _out(y, "y", (P, N), torch.bfloat16, dev)
    if P == 0 or N == 0:
        return y
    if check and status is None:
        status = _status(True, dev)
    code = _lib().moe_fp4_expert_product(a_codes.data_ptr(), a_scales.data_ptr(), _address(a_tensor_scale),
                                         w_codes.data_ptr(), w_scales.data_ptr(), _address(w_tensor_scale),
                                         expert_offsets.data_ptr(), P, E, N, cols, f, y.data_ptr(), _address(status), on)
    _done(code, status if check else None, "fp4_expert_product")
    return y


@_on_stream
def fp4_moe_forward(x, topk_ids, topk_weights, w_gate_up_codes, w_gate_up_scales, w_down_codes, w_down_scales,
                    fmt: str = "nvfp4", w_gate_up_tensor_scale: Optional[torch.Tensor] = None,
                    w_down_tensor_scale: Optional[torch.Tensor] = None, x_tensor_scale: Optional[torch.Tensor] = None,
                    h_tensor_scale: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, stream=None,
                    check: bool = True) -> torch.Tensor:
    """The expert layer with 4-bit experts and 4-bit activations, no adapters:

      y_t = sum_k w[t, k] W_down,e Q[ SiLU(W_gate,e Q[x_t]) * (W_up,e Q[x_t]) ],  e = topk_ids[t, k]

    with Q the quantisation of the activations.  x [T, H] bf16; w_gate_up_* of a
    stack [E, 2I, H] (gate rows first), w_down_* of a stack [E, H, I], quantised
    once by fp4_quantize.  Returns y bf16 [T, H]."""
    if not isinstance(x, torch.Tensor) or not isinstance(w_gate_up_codes, torch.Tensor):
        raise TypeError("x and w_gate_up_codes must be torch.Tensors")
    _req(x, "x", torch.bfloat16, x.device)
    if x.dim() != 2 or w_gate_up_codes.dim() != 3 or w_gate_up_codes.shape[1] % 2:
        raise ValueError("fp4_moe_forward: inconsistent shapes")
    E, I = w_gate_up_codes.shape[0], w_gate_up_codes.shape[1] // 2
    if w_down_codes.dim() != 3 or w_down_codes.shape[1] != x.shape[1]:
        raise ValueError("fp4_moe_forward: inconsistent shapes")
    H = x.shape[1]
    pos, offsets = moe_sort_pairs(topk_ids, E, check=check)
    a, sa = fp4_quantize_permuted(x, topk_ids, pos, offsets, fmt, x_tensor_scale)
    gu = fp4_expert_product(a, sa, offsets, w_gate_up_codes, w_gate_up_scales, H, fmt, x_tensor_scale,
                            w_gate_up_tensor_scale, check=check)
    h, sh = fp4_quantize_swiglu(gu, offsets, fmt, h_tensor_scale)
    d = fp4_expert_product(h, sh, offsets, w_down_codes, w_down_scales, I, fmt, h_tensor_scale, w_down_tensor_scale,
                           check=check)
    return moe_unpermute(d, pos, topk_weights, y=y)
