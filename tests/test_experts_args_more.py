"""More refusals of the expert operators, before any launch."""
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


@pytest.mark.parametrize("outputs", [127, 128])
def test_product_refuses_half_an_element(lib, outputs):
    """y between two bf16 elements is not an address of a bf16 tensor."""
    assert lib.moe_fp4_expert_product(FAKE, FAKE, None, FAKE, FAKE, None, FAKE, 4, 2, outputs, 64, 0, ODD, None,
                                      None) == mlr.MLR_ERR_INVALID


def calls():
    """Every entry point with tensors of the right types and shapes, on the host;
    an empty batch as well, which launches nothing."""
    E, P, N, C = 2, 8, 128, 64
    x, ids, rows, w = torch.zeros(4, C, dtype=BF), i32(4, 2), torch.zeros(8, C, dtype=BF), torch.zeros(4, 2)
    off, codes, scales = i32(E + 1), u8(P, 32), u8(P // 128 + E, 1, 32, 4, 4)
    wc, ws = u8(E, N, 32), u8(E, 1, 1, 32, 4, 4)
    dc, ds = u8(E, C, 32), u8(E, 1, 1, 32, 4, 4)
    return {
        "moe_permute": lambda: pm.moe_permute(x, ids, E),
        "moe_permute unchecked": lambda: pm.moe_permute(x, ids, E, check=False),
        "moe_permute empty": lambda: pm.moe_permute(x[:0], ids[:0], E),
        "moe_sort_pairs": lambda: pm.moe_sort_pairs(ids, E),
        "moe_permute_backward": lambda: pm.moe_permute_backward(rows, ids),
        "moe_unpermute": lambda: pm.moe_unpermute(rows, ids, w),
        "moe_unpermute empty": lambda: pm.moe_unpermute(rows[:0], ids[:0], w[:0]),
        "moe_unpermute_backward": lambda: pm.moe_unpermute_backward(x, rows, ids, w),
        "MoePermute": lambda: pm.MoePermute.apply(x, ids, E),
        "MoeUnpermute": lambda: pm.MoeUnpermute.apply(rows, ids, w),
        "fp4_quantize": lambda: fp4.fp4_quantize(x),
        "fp4_quantize_permuted": lambda: fp4.fp4_quantize_permuted(x, ids, ids, off),
        "fp4_quantize_swiglu": lambda: fp4.fp4_quantize_swiglu(torch.zeros(P, 2 * C), off),
        "fp4_dequantize": lambda: fp4.fp4_dequantize(codes, scales, C, expert_offsets=off),
        "fp4_expert_product": lambda: fp4.fp4_expert_product(codes, scales, off, wc, ws, C),
        "fp4_moe_forward": lambda: fp4.fp4_moe_forward(x, ids, w, wc, ws, dc, ds),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="must be on a CUDA device"):
        calls()[name]()


class On:
    """As much of a tensor as tells where it is."""

    def __init__(self, index):
        self.device, self.is_cuda = torch.device("cuda", index), True

    def get_device(self):
        return self.device.index


def test_tensors_of_another_device_are_refused(monkeypatch):
    """The kernels go to the current device's stream."""
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 70 + d, raising=False)
    assert mlr._launch_stream(On(1), "call") == 71
    with pytest.raises(ValueError, match="tensors are on cuda:0, .* is cuda:1"):
        mlr._launch_stream(On(0), "call")


def test_workspace_of_sorts_with_and_without_rows(lib):
    """One launch, which keeps nothing, sorts 8192 pairs with rows and 16384 without."""
    rows, order = lib.moe_permute_workspace_bytes, lib.moe_sort_pairs_workspace_bytes
    for T, K in ((1, 1), (1024, 8), (8192, 1)):
        assert rows(T, K, 60) == 1 and order(T, K, 60) == 1
    for T, K in ((1025, 8), (2048, 8), (16384, 1)):
        assert rows(T, K, 60) > 4 * 61 and order(T, K, 60) == 1
    for T, K in ((2049, 8), (16385, 1), (1 << 20, 8)):
        assert order(T, K, 60) == rows(T, K, 60) > 4 * 61
    for bad in ((-1, 2, 3), (4, 257, 3), (4, 2, 16385), (4, 2, 0)):
        assert order(*bad) == 0
