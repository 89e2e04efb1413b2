"""Calls of the norm and the router that no kernel may see, refused before any launch (CPU)."""
import ctypes

import pytest

import __graft_entry__
import lora_moe_expert_info_gb300 as mlr
from lora_moe_expert_info_gb300 import norm, router

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: the calls return before any launch
HALF = ctypes.c_void_p(0x1002)  # on no 4-byte boundary
BIG = ctypes.c_size_t(1 << 40)


@pytest.fixture(scope="module", autouse=True)
def lib():
    __graft_entry__.build()
    norm._lib(), router._lib()
    return mlr.library()


@pytest.mark.parametrize("T", [4, 4096])
@pytest.mark.parametrize("name", ["ids", "weights", "status"])
def test_choice_into_addresses_off_the_grid(lib, name, T):
    a = dict(ids=FAKE, weights=FAKE, status=None) | {name: HALF}
    assert lib.moe_route(FAKE, None, None, T, 16, 2, 1, 1, 1, 0, 1, 1.0, a["ids"], a["weights"], a["status"],
                         None) == mlr.MLR_ERR_INVALID


@pytest.mark.parametrize("T", [0, 4, 4096])
@pytest.mark.parametrize("name", ["ids", "loss", "counts", "status"])
def test_loss_into_addresses_off_the_grid(lib, name, T):
    a = dict(ids=FAKE, loss=FAKE, counts=FAKE, status=None) | {name: HALF}
    assert lib.moe_balance_loss(FAKE, a["ids"], None, T, 256, 2, 1, 0, a["loss"], a["counts"], FAKE, BIG, a["status"],
                                None) == mlr.MLR_ERR_INVALID


@pytest.mark.parametrize("name", ["ids", "d_weights", "counts", "d_loss", "status"])
def test_gradient_of_addresses_off_the_grid(lib, name):
    a = dict(ids=FAKE, d_weights=FAKE, counts=FAKE, d_loss=FAKE, status=None) | {name: HALF}
    assert lib.moe_route_backward(FAKE, a["ids"], a["d_weights"], a["counts"], a["d_loss"], None, 4, 16, 2, 1, 0, 1, 1.0,
                                  FAKE, a["status"], None) == mlr.MLR_ERR_INVALID


@pytest.mark.parametrize("codes", [None, ctypes.c_void_p(0x9000)])
def test_norm_with_one_place_for_both_outputs(lib, codes):
    """y and the new residual stream in one buffer: the second would be lost."""
    assert lib.moe_rms_norm(FAKE, FAKE, FAKE, 4, 64, 0, 0, 1e-6, FAKE, FAKE, codes, codes, None) == mlr.MLR_ERR_INVALID


def test_workspace_of_the_loss_by_tokens(lib):
    """One launch without a workspace pays only up to so many tokens, however few experts."""
    ws = lib.moe_balance_loss_workspace_bytes
    assert ws(8192, 8) == ws(8192, 64) == ws(4096, 128) == 1
    assert ws(8193, 8) > 4 * 17 and ws(65536, 8) > 4 * 17 and ws(8193, 64) > 4 * 129 and ws(8192, 65) > 4 * 131
