"""Refusals of the sort, quantisation and product calls, before any launch
(CPU tensors and never-dereferenced pointers)."""
import ctypes

import pytest
import torch

import __graft_entry__
import lora_moe_expert_info_gb300 as mlr
from lora_moe_expert_info_gb300 import fp4, permute as pm

BF = torch.bfloat16
FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module", autouse=True)
def lib():
    __graft_entry__.build()
    pm._lib(), fp4._lib()
    return mlr.library()


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def test_permute_binding_refusals():
    x, ids = torch.zeros(4, 8, dtype=BF), i32(4, 2)
    with pytest.raises(TypeError):
        pm.moe_permute(x.half(), ids, 3)
    with pytest.raises(TypeError):
        pm.moe_permute(x, ids.long(), 3)
    with pytest.raises(TypeError):
        pm.moe_permute(None, ids, 3)
    with pytest.raises(ValueError):
        pm.moe_permute(x[:3], ids, 3)
    with pytest.raises(ValueError):
        pm.moe_permute(x.t(), ids, 3)  # not contiguous
    with pytest.raises(ValueError):
        pm.moe_permute(x, ids, 0)
    with pytest.raises(ValueError):
        pm.moe_permute(x, ids.view(-1), 3)
    with pytest.raises(ValueError):
        pm.moe_permute(x, ids, 3, rows=torch.zeros(7, 8, dtype=BF))
    with pytest.raises(ValueError):
        pm.moe_sort_pairs(ids, 16385)
    rows, w = torch.zeros(8, 8, dtype=BF), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        pm.moe_unpermute(rows[:6], ids, w)
    with pytest.raises(TypeError):
        pm.moe_unpermute(rows, ids, w.double())
    with pytest.raises(TypeError):
        pm.moe_unpermute(rows, ids, None)
    with pytest.raises(TypeError):
        pm.moe_unpermute_backward(x.float(), rows, ids, w)
    with pytest.raises(ValueError):
        pm.moe_unpermute_backward(x[:3], rows, ids, w)


def test_permute_abi_refusals(lib):
    ws = lib.moe_permute_workspace_bytes(4, 2, 3)
    assert ws > 0 and lib.moe_permute_workspace_bytes(-1, 2, 3) == 0 and lib.moe_permute_workspace_bytes(4, 257, 3) == 0
    f = lib.moe_permute
    assert f(FAKE, FAKE, 4, 2, 8, 3, 0, None, FAKE, FAKE, FAKE, ws, None, None) == mlr.MLR_ERR_INVALID
    assert f(FAKE, FAKE, 4, 2, 8, 3, 7, FAKE, FAKE, FAKE, FAKE, ws, None, None) == mlr.MLR_ERR_INVALID
    assert f(FAKE, FAKE, 4, 2, 0, 3, 0, FAKE, FAKE, FAKE, FAKE, ws, None, None) == mlr.MLR_ERR_INVALID
    assert f(ODD, FAKE, 4, 2, 8, 3, 0, FAKE, FAKE, FAKE, FAKE, ws, None, None) == mlr.MLR_ERR_INVALID
    assert f(FAKE, FAKE, 4, 2, 8, 3, 0, FAKE, FAKE, FAKE, FAKE, ws - 1, None, None) == mlr.MLR_ERR_CAPACITY
    assert f(FAKE, FAKE, 1 << 30, 2, 8, 3, 0, FAKE, FAKE, FAKE, FAKE, ws, None, None) == mlr.MLR_ERR_UNSUPPORTED
    assert lib.moe_unpermute(FAKE, FAKE, FAKE, 4, 2, 8, 2, FAKE, None, None) == mlr.MLR_ERR_INVALID
    assert lib.moe_unpermute(None, FAKE, FAKE, 4, 2, 8, 0, FAKE, None, None) == mlr.MLR_ERR_INVALID
    assert lib.moe_unpermute(FAKE, FAKE, FAKE, 0, 2, 8, 0, FAKE, None, None) == mlr.MLR_OK
    assert lib.moe_unpermute_backward(FAKE, FAKE, FAKE, None, 4, 2, 8, 0, FAKE, FAKE, None, None) == mlr.MLR_ERR_INVALID


def test_quantize_binding_refusals():
    x = torch.zeros(4, 64, dtype=BF)
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x, "fp4")
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x, "mxfp4", torch.ones(1))
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x, "nvfp4", torch.ones(2))
    with pytest.raises(TypeError):
        fp4.fp4_quantize(x, "nvfp4", torch.ones(1, dtype=torch.float64))
    with pytest.raises(TypeError):
        fp4.fp4_quantize(x.half())
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x[0])
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x[:, :0])
    with pytest.raises(ValueError):
        fp4.fp4_quantize(x, codes=u8(4, 16))
    ids, off = i32(4, 2), i32(4)
    with pytest.raises(ValueError):
        fp4.fp4_quantize_permuted(x, ids, ids[:3], off)
    with pytest.raises(TypeError):
        fp4.fp4_quantize_permuted(x, ids, ids, off.long())
    with pytest.raises(ValueError):
        fp4.fp4_quantize_permuted(x, ids, ids, off[:1])
    with pytest.raises(ValueError):
        fp4.fp4_quantize_swiglu(x[:, :63].contiguous(), off)
    with pytest.raises(ValueError):
        fp4.fp4_dequantize(u8(4, 32), u8(1, 1, 32, 4, 4), 96, "nvfp4")
    with pytest.raises(TypeError):
        fp4.fp4_dequantize(u8(4, 32), u8(1, 1, 32, 4, 4), 64, "nvfp4", dtype=torch.float16)


def test_product_binding_refusals():
    E, N, C, P = 2, 130, 64, 5
    off, a, sa = i32(E + 1), u8(P, 32), u8(P // 128 + E, 1, 32, 4, 4)
    w, sw = u8(E, N, 32), u8(E, 2, 1, 32, 4, 4)
    f = fp4.fp4_expert_product
    with pytest.raises(ValueError):
        f(a, sa, off, w, sw, 65, "nvfp4")
    with pytest.raises(ValueError):
        f(a, sa[:1], off, w, sw, C, "nvfp4")
    with pytest.raises(ValueError):
        f(a, sa, off, w[:1], sw, C, "nvfp4")
    with pytest.raises(ValueError):
        f(a, sa, off, w, sw[:, :1].contiguous(), C, "nvfp4")
    with pytest.raises(ValueError):
        f(a, sa, off, w, sw, C, "mxfp4", torch.ones(1))
    with pytest.raises(ValueError):
        f(a, sa, off, w, sw, C, "nvfp4", None, torch.ones(1))
    with pytest.raises(TypeError):
        f(a.to(torch.int8), sa, off, w, sw, C)
    with pytest.raises(ValueError):
        f(a, sa, off, w, sw, C, y=torch.zeros(P, N + 1, dtype=BF))


def test_fp4_abi_refusals(lib):
    assert lib.moe_fp4_pitch(1) == 16 and lib.moe_fp4_pitch(33) == 32 and lib.moe_fp4_pitch(0) == -1
    assert lib.moe_fp4_scale_atoms(65, 1) == 2 and lib.moe_fp4_scale_atoms(65, 0) == 1
    assert lib.moe_fp4_scale_atoms(65, 2) == -1
    q = lib.moe_fp4_quantize
    assert q(FAKE, 1, 4, 64, 0, 2, None, FAKE, FAKE, None) == mlr.MLR_ERR_INVALID
    assert q(FAKE, 1, 4, 64, 0, 0, FAKE, FAKE, FAKE, None) == mlr.MLR_ERR_INVALID
    assert q(FAKE, 1, 4, 64, 0, 0, None, ODD, FAKE, None) == mlr.MLR_ERR_INVALID
    assert q(FAKE, 1, 4, (1 << 19) + 1, 0, 0, None, FAKE, FAKE, None) == mlr.MLR_ERR_UNSUPPORTED
    assert q(FAKE, 1, 0, 64, 0, 0, None, FAKE, FAKE, None) == mlr.MLR_OK
    f = lib.moe_fp4_quantize_permuted
    assert f(FAKE, None, FAKE, FAKE, 4, 2, 64, 3, 0, 0, None, FAKE, FAKE, None, None) == mlr.MLR_ERR_INVALID
    assert f(FAKE, FAKE, FAKE, FAKE, 4, 513, 64, 3, 0, 0, None, FAKE, FAKE, None, None) == mlr.MLR_ERR_UNSUPPORTED
    g = lib.moe_fp4_quantize_swiglu
    assert g(FAKE, None, 4, 64, 3, 0, 0, None, FAKE, FAKE, None, None) == mlr.MLR_ERR_INVALID
    p = lib.moe_fp4_expert_product
    ok = [FAKE, FAKE, None, FAKE, FAKE, None, FAKE, 4, 2, 128, 64, 0, FAKE, None, None]
    for i, v, code in ((0, None, mlr.MLR_ERR_INVALID), (3, ODD, mlr.MLR_ERR_INVALID), (2, FAKE, mlr.MLR_ERR_INVALID),
                       (6, None, mlr.MLR_ERR_INVALID), (8, 0, mlr.MLR_ERR_INVALID), (8, 16385, mlr.MLR_ERR_UNSUPPORTED),
                       (9, 0, mlr.MLR_ERR_INVALID), (11, 5, mlr.MLR_ERR_INVALID), (12, None, mlr.MLR_ERR_INVALID),
                       (7, 0, mlr.MLR_OK)):
        args = list(ok)
        args[i] = v
        assert p(*args) == code, (i, v)
