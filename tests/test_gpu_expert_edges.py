"""Corners of the expert operators' arguments: buffers at every address their type
allows."""
import math

import pytest
import torch

from lora_moe_expert_info_gb300 import fp4
from test_gpu_fp4 import FMTS, product_case

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,K,E,N,C,masked", [(1, 8, 16, 2, 64, 0.0), (40, 2, 3, 130, 96, 0.2), (40, 2, 3, 129, 96, 0.2),
                                              (700, 1, 2, 256, 320, 0.1), (513, 2, 3, 71, 128, 0.0)])
def test_product_into_any_address(cuda_device, fmt, T, K, E, N, C, masked):
    """y at every address a bf16 tensor may begin at, NaN around it: the same
    results as at a 512-byte boundary, and nothing around y is written.  Few rows
    per expert and many, outputs even and odd, rows past the last expert's."""
    off, a, sa, qw, sw, ga, gw = product_case(T, K, E, N, C, fmt, seed=N, masked=masked)
    want = fp4.fp4_expert_product(a, sa, off, qw, sw, C, fmt, ga, gw)
    n = T * K * N
    for k in range(9):
        buf = torch.full((n + 32,), math.nan, dtype=BF, device="cuda")
        y = buf[k:k + n].view(T * K, N)
        out = fp4.fp4_expert_product(a, sa, off, qw, sw, C, fmt, ga, gw, y=y)
        assert out is y and torch.equal(y, want), k
        assert buf[:k].isnan().all() and buf[k + n:].isnan().all(), k
