"""More refusals of the expert operators, before any launch."""
import ctypes

import pytest

import __graft_entry__
import lora_moe_expert_info_gb300 as mlr
from lora_moe_expert_info_gb300 import fp4, permute as pm

FAKE = ctypes.c_void_p(0x1000)
ODD = ctypes.c_void_p(0x1001)


@pytest.fixture(scope="module", autouse=True)
def lib():
    __graft_entry__.build()
    pm._lib(), fp4._lib()
    return mlr.library()


@pytest.mark.parametrize("outputs", [127, 128])
def test_product_refuses_half_an_element(lib, outputs):
    """y between two bf16 elements is not an address of a bf16 tensor."""
    assert lib.moe_fp4_expert_product(FAKE, FAKE, None, FAKE, FAKE, None, FAKE, 4, 2, outputs, 64, 0, ODD, None,
                                      None) == mlr.MLR_ERR_INVALID
