"""The norm at the ends of float32's range, against 64 bits.

Tolerance: that of the ordinary rows, (u + (H / 2 + 8) 2^-24) |y| with u half a step of the
output's type, and near its smallest numbers half a step of these (bf16 2^-134, float32
2^-150) of the result and, at most twice as much, of float32's product before it.
"""
import math

import numpy as np
import pytest
import torch

from lora_moe_expert_info_gb300 import norm
from oracle import router as ox

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U, LEAST = {BF: 2.0 ** -8, F32: 2.0 ** -24}, {BF: 2.0 ** -134 + 2.0 ** -149, F32: 3 * 2.0 ** -150}


def f64(t):
    return t.detach().cpu().double().numpy()


# one element, off and on the 16-byte grid, all units a thread, eight and four to a vector
@pytest.mark.parametrize("H", [1, 65, 128, 520, 1111, 2048, 4099, 7168, 8200, 16384])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("w_dtype", [BF, F32])
@pytest.mark.parametrize("rows", [3, 1100])
def test_weights_of_infinity(cuda_device, H, dtype, w_dtype, rows):
    """A weight of infinity gives infinities of the elements' signs (NaN times 0), and leaves
    the other columns as they are."""
    g = torch.Generator().manual_seed(H)
    x = torch.randn(rows, H, generator=g).to(dtype).cuda()
    w = torch.randn(H, generator=g).to(w_dtype).cuda()
    plain, _ = norm.rms_norm(x, w)
    at = torch.arange(0, H, 3, device="cuda")
    w[at[::2]], w[at[1::2]] = math.inf, -math.inf
    if H > 9:
        w[7] = math.nan
        x[0, 0] = 0
    y, _ = norm.rms_norm(x, w)
    want = x.double() * w.double()
    assert torch.equal(y[:, at].isnan(), want[:, at].isnan())
    assert torch.equal(y[:, at].nan_to_num(5, 9, -9), want[:, at].nan_to_num(5, 9, -9).to(dtype))
    if H > 9:
        assert y[:, 7].isnan().all()
        rest = torch.ones(H, dtype=torch.bool, device="cuda")
        rest[at], rest[7] = False, False
        assert torch.equal(y[1:, rest], plain[1:, rest])


@pytest.mark.parametrize("H", [1, 65, 128, 1111, 2048, 7168, 16384])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("w_dtype", [BF, F32])
def test_products_beyond_the_range_of_a_times_w(cuda_device, H, dtype, w_dtype):
    """Rows of 2^-60 to 2^55 and weights of 2^-120 to 2^120: y = r m w is in the range where r
    times w alone is not, or is below its normal numbers."""
    g = torch.Generator().manual_seed(H)
    for rows in (2.0 ** -60, 2.0 ** -39, 2.0 ** -20, 1.0, 2.0 ** 20, 2.0 ** 39, 2.0 ** 55):
        for size in (2.0 ** -120, 2.0 ** -95, 1.0, 2.0 ** 95, 2.0 ** 120):
            x = (torch.randn(5, H, generator=g) * rows).to(dtype).cuda()
            w = ((1 + torch.rand(H, generator=g)) * size).to(w_dtype).cuda()
            y, _ = norm.rms_norm(x, w, 0.0)
            want = ox.norm(f64(x), f64(w), 0.0)
            assert np.all(np.abs(f64(y) - want) <= (U[dtype] + (H / 2 + 8) * 2.0 ** -24) * np.abs(want) + LEAST[dtype])
