"""The router's operators at the ends of float32's range, against 64 bits.

Tolerances.  expf is within two units of the last place of its result, 2^-22 of it, or
2^-148 where that is below the normal numbers; a sigmoid e / (1 + e) adds two roundings of
2^-24 each (2^-150 below the normal numbers).
"""
import math

import numpy as np
import pytest
import torch

from lora_moe_expert_info_gb300 import router as rt
from oracle import router as ox

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().double().numpy()


# the kernel of eight and of sixteen places, rows off the 16-byte grid, the one for many experts or places
KINDS = [(64, 8), (256, 8), (130, 6), (512, 12), (61, 3), (1100, 4), (96, 20)]


@pytest.mark.parametrize("E,K", KINDS)
@pytest.mark.parametrize("scale", [1.0, 2.5, 16.0])
def test_weights_of_the_smallest_sigmoids(cuda_device, E, K, scale):
    """Renormalised weights and their gradients where all sigmoids of a token are next to
    nothing: a few open experts with logits from -60 to -89."""
    T = 300
    rng = np.random.default_rng(E)
    l = np.full((T, E), -np.inf, np.float32)
    for t in range(T):
        n = (1, 2, K, K + 2)[t % 4]
        l[t, rng.permutation(E)[:n]] = -60 - 29 * t / (T - 1) + rng.random(n) * (t % 3)
    l = np.maximum(l, np.where(np.isfinite(l), -89, -np.inf)).astype(np.float32)
    lt = torch.from_numpy(l).cuda()
    ids, w = rt.moe_route(lt, K, "sigmoid", scale=scale)
    ref = ox.choose(l.astype(float), K, "sigmoid")
    assert np.array_equal(ids.cpu().numpy(), ref)
    s = (ox.taken(ref, E, l) * ox.scores(l.astype(float), "sigmoid")[:, None, :]).sum(2)
    total = s.sum(1, keepdims=True)
    rw = scale * s / total
    least = np.where(s > 0, s, 1).min(1, keepdims=True)
    # each sigmoid as above, their sum, the quotient and the scale: K + 4 roundings
    eps = 2 * (2.0 ** -22 + 2.0 ** -23 + (2.0 ** -148 + 2.0 ** -149) / least) + (K + 4) * 2.0 ** -24
    assert np.all(np.abs(f64(w) - rw) <= eps * rw)
    g = rng.normal(size=(T, K)).astype(np.float32)
    d = rt.moe_route_backward(lt, ids, torch.from_numpy(g).cuda(), scoring="sigmoid", scale=scale)
    rd = ox.weights_backward(g.astype(float), l.astype(float), ref, "sigmoid", True, scale)
    mag = 2 * scale * np.abs(g).sum(1, keepdims=True)  # a weight's share is at most 1
    assert np.all(np.abs(f64(d) - rd) <= (eps + 4 * 2.0 ** -24) * mag)
