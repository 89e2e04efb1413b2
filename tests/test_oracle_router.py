"""The oracle's norm, choice, loss and gradients against differences, worked
examples and torch's own numbers, on the CPU."""
import numpy as np
import pytest
import torch

from oracle import router as ox


def difference(f, x, h=1e-5):
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        out[i] = (f(a) - f(b)) / (2 * h)
    return out


def test_norm_gradient_is_that_of_the_norm():
    rng = np.random.default_rng(0)
    r, w, dy, d_r = rng.normal(size=(3, 5)), rng.normal(size=5), rng.normal(size=(3, 5)), rng.normal(size=(3, 5))
    dx, dw, _, _ = ox.norm_backward(dy, r, w, 1e-2, d_r)
    assert np.allclose(dx, difference(lambda v: (ox.norm(v, w, 1e-2) * dy).sum() + (v * d_r).sum(), r), atol=1e-8)
    assert np.allclose(dw, difference(lambda v: (ox.norm(r, v, 1e-2) * dy).sum(), w), atol=1e-8)


def test_eight_bits_are_those_of_torch():
    assert len(ox.E4M3) == 127 and ox.E4M3[-1] == 448
    assert np.array_equal(ox.E4M3, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    rng = np.random.default_rng(1)
    y = (rng.normal(size=(4, 300)) * np.exp(rng.normal(size=(4, 300)) * 3)).astype(np.float32).astype(float)
    y[1, 128:256] = 0
    y[2, 5] = 448 * 2.0 ** 3  # the group's largest, on the border
    codes, exps = ox.eight_bits(y)
    assert exps[1, 1] == 127 and exps[2, 0] == 130
    s = np.repeat(exps.astype(int), 128, axis=1)[:, :300] - 127
    ref = torch.from_numpy((y * 2.0 ** -s).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, ref)
    assert np.all(np.abs(ox.from_eight_bits(codes, exps) - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** (s - 10.0)))


def test_choice_worked_by_hand():
    l = np.array([[0.0, 2.0, 2.0, -np.inf, 1.0, np.nan]])
    assert ox.choose(l, 4, "softmax").tolist() == [[1, 2, 4, 0]]
    assert ox.choose(l, 6, "softmax").tolist() == [[1, 2, 4, 0, -1, -1]]
    # groups {0, 2}, {2, none}, {1, none}: best experts 2, 2, 1
    assert ox.choose(l, 2, "softmax", groups=3, best=1).tolist() == [[1, 0]]
    # sums of two: 0.5 + s(2), s(2), s(1): the first, then the second group
    assert ox.choose(l, 3, "sigmoid", groups=3, best=2).tolist() == [[1, 2, 0]]
    assert ox.choose(l, 2, "sigmoid", bias=np.array([1.0, 0, 0, 9, 0, 9])).tolist() == [[0, 1]]
    assert ox.choose(l, 2, "softmax", mask=np.array([False])).tolist() == [[-1, -1]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_weight_and_loss_gradients(scoring, renormalize):
    rng = np.random.default_rng(2)
    l = rng.normal(size=(4, 6))
    ids = ox.choose(l, 3, scoring)
    ids[1, 2] = -1
    ids[2, 1] = ids[2, 0]  # the same expert twice
    g = rng.normal(size=(4, 3))
    want = difference(lambda v: (ox.weights(v, ids, scoring, renormalize, 2.5) * g).sum(), l)
    assert np.allclose(ox.weights_backward(g, l, ids, scoring, renormalize, 2.5), want, atol=1e-8)
    mask = np.array([True, True, False, True])
    loss, counts = ox.balance(l, ids, scoring, mask)
    assert counts[-1] == 3 and counts[:-1].sum() == 8
    want = difference(lambda v: 0.7 * ox.balance(v, ids, scoring, mask)[0], l)
    assert np.allclose(ox.balance_backward(0.7, l, counts, 3, scoring, mask), want, atol=1e-8)


def test_even_use_has_loss_one():
    E, K = 8, 2
    ids = np.arange(16).reshape(8, 2) % E
    assert abs(ox.balance(np.zeros((8, E)), ids, "softmax")[0] - 1) < 1e-12
    assert abs(ox.balance(np.zeros((8, E)), ids, "sigmoid")[0] - 1) < 1e-12
