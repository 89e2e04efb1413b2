"""The restatements of the expert sort and the 4-bit formats, pinned on CPU
against worked values and the definitions."""
import numpy as np
import pytest
import torch

from oracle import experts as ox


def test_sort_worked_example():
    ids = np.array([[2, 0], [0, -1], [2, 2]], dtype=np.int32)
    pos, off = ox.sort_pairs(ids, 3)
    assert pos.tolist() == [[2, 0], [1, ~5], [3, 4]]
    assert off.tolist() == [0, 2, 2, 5]


def test_e2m1_ties_and_saturation():
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert [ox.round_e2m1(t) for t in ties] == [0, 2, 2, 4, 4, 6, 6]
    assert [ox.round_e2m1(np.nextafter(t, 9)) for t in ties] == [1, 2, 3, 4, 5, 6, 7]
    assert [ox.round_e2m1(np.nextafter(t, 0)) for t in ties] == [0, 1, 2, 3, 4, 5, 6]
    assert ox.round_e2m1(1e9) == 7


def test_e4m3_rounding_matches_the_float8_cast():
    v = torch.cat([torch.linspace(0, 448, 5001), torch.logspace(-4, 2, 3001)]).clamp(max=448)
    want = v.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert [ox.round_e4m3(float(x)) for x in v] == want.tolist()


@pytest.mark.parametrize("most,s", [(6.0, 0), (np.nextafter(np.float32(6), np.float32(7)), 1), (3.0, -1), (0.0, 0),
                                    (1e-40, -127), (3.4e38, 126)])
def test_mx_scale_is_the_smallest_that_covers(most, s):
    byte, val, r = ox.block_scale(float(most), "mxfp4")
    assert byte == s + 127 and val == 2.0 ** s and r == 2.0 ** -s
    assert float(most) <= 6 * val


def test_nv_scale_of_a_calibrated_matrix_reaches_448():
    byte, val, _ = ox.block_scale(2688.0 * 0.125, "nvfp4", 0.125)
    assert byte == 0x7E and val == 56.0


def test_quantized_value_is_the_nearest():
    rng = np.random.default_rng(0)
    x = rng.standard_normal(64).astype(np.float32)
    for fmt, n in (("mxfp4", 32), ("nvfp4", 16)):
        codes, byts, vals = ox.quantize_row(x, fmt)
        got = ox.code_values(codes) * np.repeat(vals, n)
        grid = np.concatenate([ox.E2M1, -ox.E2M1])
        best = np.abs(np.repeat(vals, n)[:, None] * grid - x[:, None]).min(1)
        assert np.all(np.abs(got - x) <= best * (1 + 1e-6))


def test_bad_blocks_are_nan_with_zero_codes():
    x = np.zeros(48, dtype=np.float32)
    x[3], x[40] = np.inf, np.nan
    codes, byts, vals = ox.quantize_row(x, "nvfp4")
    assert byts.tolist() == [0x7F, 0, 0x7F] and not codes.any() and np.isnan(vals[0])
    codes, byts, vals = ox.quantize_row(x, "mxfp4")
    assert byts.tolist() == [0xFF, 0xFF] and not codes.any()
