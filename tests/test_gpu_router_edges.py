"""The router's operators at the ends of float32's range, against 64 bits.

Tolerances.  expf is within two units of the last place of its result, 2^-22 of it, or
2^-148 where that is below the normal numbers; a sigmoid e / (1 + e) adds two roundings of
2^-24 each (2^-150 below the normal numbers).
"""
import math

import numpy as np
import pytest
import torch

from lora_moe_expert_info_gb300 import norm, router as rt
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


@pytest.mark.parametrize("E,G,K", [(32, 4, 4), (256, 8, 8), (130, 10, 6), (512, 16, 16), (48, 3, 20)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_groups_whose_sums_pass_the_range_downwards(cuda_device, E, G, K, dtype):
    """Biases that push all experts of some groups so far away that two scores add up to
    less than float32's lowest: those groups still have an order, above the empty ones."""
    T, size = 40, E // G
    rng = np.random.default_rng(E)
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(E)).to(dtype).cuda()
    l[1::4, :size] = -math.inf                     # an empty group before all others
    l[2::4, 2 * size:2 * size + size] = -math.inf  # one among them
    l[3::4, 1:size] = -math.inf                    # a group of one expert
    lowest = float(np.finfo(np.float32).min)
    for case in range(5):
        b = -(1.8e38 + 1.5e38 * rng.random(E))     # all groups beyond the range
        if case == 1:
            b[:size], b[size:2 * size] = -3.0e38, -2.0e38
        elif case == 2:
            b[:] = lowest                          # of equal scores the lowest index
        elif case == 3:
            b[-size:] = 0.1 * rng.random(size)     # one group within it
        elif case == 4:
            b[size:2 * size] = 1.9e38              # one beyond it upwards
        bias = torch.from_numpy(b.astype(np.float32)).cuda()
        for best in range(-(-K // size), G):
            ids, w = rt.moe_route(l, K, "sigmoid", bias, G, best)
            ref = ox.choose(f64(l), K, "sigmoid", f64(bias), G, best)
            assert np.array_equal(ids.cpu().numpy(), ref), (case, best)
            assert torch.isfinite(w).all()


def complement(l):
    """1 - sigmoid, without the difference."""
    return ox.sigmoid(-l)


@pytest.mark.parametrize("E,K", KINDS)
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradients_of_sigmoids_near_one(cuda_device, E, K, renormalize):
    """Logits of 8 to 80: the gradients have the factor 1 - sigmoid, which is far below the
    last place of the sigmoid, and are right relative to themselves."""
    T = 200
    rng = np.random.default_rng(E)
    l = rng.uniform(8, np.linspace(9, 80, T)[:, None], (T, E)).astype(np.float32)
    l[:, ::3] *= -1
    lt = torch.from_numpy(l).cuda()
    ids, _ = rt.moe_route(lt, K, "sigmoid")
    idn, ln = ids.cpu().numpy(), l.astype(float)
    g = rng.normal(size=(T, K)).astype(np.float32)
    near, gd = np.take_along_axis(complement(ln), idn, 1), g.astype(float)
    s = np.take_along_axis(ox.sigmoid(ln), idn, 1)
    if renormalize:
        share = s / s.sum(1, keepdims=True)
        part = 2.5 * share * (gd - (gd * share).sum(1, keepdims=True)) * near
        mag = 2.5 * share * (np.abs(gd) + (np.abs(gd) * share).sum(1, keepdims=True)) * near
    else:
        part = 2.5 * gd * s * near
        mag = np.abs(part)
    want, room = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(want, idn, part, 1)
    np.put_along_axis(room, idn, mag, 1)
    # a share: exponential and quotient 6, divisor 6 + K, 2 more; the mean of K shares 14 + 2 K;
    # the complement 6, products 4
    eps = (3 * K + 40) * 2.0 ** -24
    d = rt.moe_route_backward(lt, ids, torch.from_numpy(g).cuda(), scoring="sigmoid", renormalize=renormalize, scale=2.5)
    assert np.all(np.abs(f64(d) - want) <= eps * room + 2.0 ** -140)
    # the loss's: p (1 - s) (a - sum p a)
    loss, counts = rt.moe_balance_loss(lt, ids, "sigmoid")
    one = torch.tensor([0.7], device="cuda")
    a = float(one) * f64(counts)[:E] * E / (K * T * T)
    p = ox.sigmoid(ln) / ox.sigmoid(ln).sum(1, keepdims=True)
    want = p * complement(ln) * (a - (p * a).sum(1, keepdims=True))
    room = p * complement(ln) * (a + (p * a).sum(1, keepdims=True))
    # the same with sums over E experts, and reciprocals a unit of the last place off
    eps = (3 * E + 56) * 2.0 ** -24
    d = rt.moe_route_backward(lt, ids, counts=counts, d_loss=one, scoring="sigmoid")
    assert np.all(np.abs(f64(d) - want) <= eps * room + 2.0 ** -140)


@pytest.mark.parametrize("T,K", [(7, 3), (1531, 3), (12347, 7), (300001, 5), (1000003, 1)])
def test_coefficients_of_the_loss_are_rounded_once(cuda_device, T, K):
    """Two experts with equal logits and every pair with the first: its gradient is exactly a
    quarter of d_loss c E / (K N^2), in one rounding (2^-24) of that number.  Its two factors
    are held to 2^-44; the rest (2 a / 4, halves of 1) is exact."""
    l = torch.full((T, 2), 0.75, device="cuda")
    ids = torch.zeros(T, K, dtype=torch.int32, device="cuda")
    _, counts = rt.moe_balance_loss(l, ids)
    assert counts.tolist() == [T * K, 0, T]
    for v in (0.01, 0.3, 1.0, 1.7, 1e-20, 3e20):
        one = torch.tensor([v], device="cuda")
        d = f64(rt.moe_route_backward(l, ids, counts=counts, d_loss=one))
        want = float(one) * T * K * 2 / (K * float(T) * T) / 4
        assert np.all(np.abs(d[:, 0] - want) <= 2.0 ** -24 * (1 + 2.0 ** -10) * want) and np.array_equal(d[:, 1], -d[:, 0])


@pytest.mark.parametrize("E,log_T,dtype", [(2, 27, BF), (3, 26, F32), (8, 26, BF), (64, 22, F32)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_shares_of_very_many_tokens(cuda_device, E, log_T, dtype, scoring):
    """Rows of one kind, as padding gives, where every addition is rounded the same way: with
    all pairs of expert 0 the loss is E times its share.  A sum of a thread takes 64 shares
    at a time, and there are then at most T / 2^16 + 64 of these, of warps and of blocks."""
    T = 1 << log_T
    row = torch.linspace(0.3, -0.9, E).to(dtype)
    l = row.cuda().expand(T, E).contiguous()
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    loss, counts = rt.moe_balance_loss(l, ids, scoring)
    assert int(counts[0]) == T == int(counts[-1])
    s = ox.scores(f64(row)[None], scoring)[0]
    want = E * s[0] / s.sum()
    assert abs(float(loss) - want) <= (64 + T / 2 ** 16 / 16 + 64 + E + 24) * 2.0 ** -24 * want


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,K", [(4, 3), (8, 8), (64, 16), (6, 2), (1100, 3), (40, 20)])
def test_far_below_the_largest(cuda_device, E, K, dtype):
    """Weights, shares and gradients of logits up to 86 below the row's largest, at whole
    numbers so that the differences are exact: right relative to themselves, whose error is
    the exponential's few units of the last place, not one that grows with the difference."""
    T = 87
    rng = np.random.default_rng(E + K)
    l = np.full((T, E), -np.inf)
    for t in range(T):
        at = rng.permutation(E)[:K]
        l[t, at] = 20 - rng.integers(0, t + 1, K)
        l[t, at[0]], l[t, at[1]] = 20.0, 20.0 - t
    lt = torch.from_numpy(l).to(dtype).cuda()
    # in units of 2^-24: an exponential 5, a sigmoid from it 9 (1 + e 1, reciprocal 2, product 1);
    # the divisor's K terms K + 9; quotient, scale and final sum 2: K + 20
    eps = (2 * K + 20) * 2.0 ** -24
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    for renormalize in (True, False):
        ids, w = rt.moe_route(lt, K, renormalize=renormalize, scale=2.5)
        ref = ox.choose(l, K, "softmax")
        assert np.array_equal(ids.cpu().numpy(), ref)
        rw = ox.weights(l, ref, "softmax", renormalize, 2.5)
        assert np.all(np.abs(f64(w) - rw) <= eps * rw)
    # the loss of a token's smallest expert alone, by itself: 1 token, its share
    for t in range(0, T, 9):
        for scoring in ("softmax", "sigmoid"):
            row = l[t:t + 1] - (20 if scoring == "sigmoid" else 0)
            rowt = torch.from_numpy(row).to(dtype).cuda()
            low = int(np.where(np.isfinite(row[0]), row[0], 1e9).argmin())
            one = torch.full((1, 1), low, dtype=torch.int32, device="cuda")
            loss, counts = rt.moe_balance_loss(rowt, one, scoring)
            want, rc = ox.balance(row, np.array([[low]]), scoring)
            assert abs(float(loss) - want) <= eps * want
            dl = torch.ones(1, device="cuda")
            d = f64(rt.moe_route_backward(rowt, one, counts=counts, d_loss=dl, scoring=scoring))
            rd = ox.balance_backward(1.0, row, rc, 1, scoring)
            # of p (a - p_low a) [(1 - s)]: the others' gradients are p times p_low
            assert np.all(np.abs(d - rd) <= (half + 2 * eps) * np.abs(rd) + 2.0 ** -133 + 2 * (half + 2 * eps) * want * ox.scores(row, scoring))


@pytest.mark.parametrize("E", [16, 61, 256, 1100])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_masked_tokens_under_an_infinite_gradient(cuda_device, E, scoring):
    """A loss scale that ran over leaves zeros in masked tokens."""
    l = torch.randn(50, E, generator=torch.Generator().manual_seed(0)).cuda()
    mask = torch.arange(50, device="cuda") % 3 != 1
    ids, w = rt.moe_route(l, 4, scoring, token_mask=mask)
    _, counts = rt.moe_balance_loss(l, ids, scoring, mask)
    for v in (math.inf, math.nan, 3e38):
        bad = torch.full((1,), v, device="cuda")
        for g in (None, w, torch.full_like(w, v)):
            for renormalize in (True, False):
                d = rt.moe_route_backward(l, ids, g, counts, bad, scoring, renormalize, 1.0, mask)
                assert not d[~mask].any() and (v == 3e38 or not torch.isfinite(d[mask]).all())


@pytest.mark.parametrize("E,dtype", [(1024, BF), (1020, BF), (1024, F32)])
def test_offsets_beyond_32_bits(cuda_device, E, dtype):
    """More than 2^31 logits through the kernels of up to 1024 experts: the last tokens come
    out as they do alone."""
    T, K = (1 << 31) // E + 5, 4
    l = torch.zeros(T, E, dtype=dtype, device="cuda")
    tail = torch.randn(7, E, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    l[-7:] = tail
    assert l.numel() > 1 << 31
    bias = torch.linspace(0, 0.1, E, device="cuda")
    for scoring, b, G, best in (("softmax", None, 1, 1), ("sigmoid", bias, 4, 2)):
        ids, w = rt.moe_route(l, K, scoring, b, G, best, token_mask=None)
        i2, w2 = rt.moe_route(tail, K, scoring, b, G, best)
        assert torch.equal(ids[-7:], i2) and torch.equal(w[-7:], w2)
        assert (ids[:-7] == ids[0]).all() and (w[:-7] == w[0]).all()
        loss, counts = rt.moe_balance_loss(l, ids, scoring)
        of_tail = torch.bincount(i2.flatten().long(), minlength=E)
        first = torch.zeros(E, dtype=torch.long, device="cuda")
        first[ids[0].long()] = T - 7
        assert int(counts[-1]) == T and torch.equal(counts[:-1].long(), first + of_tail)
        assert abs(float(loss) - 1) < 1e-2  # all but seven tokens use every expert alike
        one = torch.ones(1, device="cuda")
        d = rt.moe_route_backward(l, ids, w, counts, one, scoring)
        assert torch.equal(d[-7:], rt.moe_route_backward(tail, i2, w2, counts, one, scoring))
        assert (d[:-7] == d[0]).all()
        del d


@pytest.mark.parametrize("T,E", [(8192, 8), (8193, 8), (65536, 8), (16384, 32), (8193, 61), (4096, 128)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_loss_with_and_without_a_workspace(cuda_device, T, E, scoring):
    """Up to 2^19 logits in one launch and in two, chosen by the workspace given."""
    K = 3
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(E)).cuda()
    ids, _ = rt.moe_route(l, K, scoring)
    loss, counts = rt.moe_balance_loss(l, ids, scoring)
    out = torch.zeros((), device="cuda"), torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    code = rt._lib().moe_balance_loss(l.data_ptr(), ids.data_ptr(), None, T, E, K, 1, rt.SCORING[scoring], out[0].data_ptr(),
                                      out[1].data_ptr(), None, 0, None, torch.cuda.current_stream().cuda_stream)
    assert code == 0
    ref, rc = ox.balance(f64(l), ids.cpu().numpy(), scoring)
    # sums of T / 64 + 64 shares at most, of warps and blocks; over experts; ten roundings of each share
    room = (T / 64 + 64 + 64 + E + 10) * 2.0 ** -24 * ref
    for a, c in ((loss, counts), out):
        assert np.array_equal(c.cpu().numpy(), rc) and abs(float(a) - ref) <= room


def test_a_training_step_from_one_graph(cuda_device):
    """Norm, router product, choice with its loss, and their gradients captured together and
    replayed on another batch with more padding, against the same step run eagerly."""
    T, H, E, K = 96, 256, 32, 4
    g = torch.Generator().manual_seed(0)
    x, res, up = (torch.randn(T, H, generator=g).cuda() for _ in range(3))
    gain, gate = torch.randn(H, generator=g).cuda().requires_grad_(), (torch.randn(H, E, generator=g) / 16).cuda().requires_grad_()
    mask = torch.arange(T, device="cuda") < 90

    def step():
        y, r = norm.RmsNorm.apply(x, gain, 1e-6, res)
        w, _, loss, _ = rt.MoeRoute.apply(y @ gate, K, "sigmoid", None, 8, 4, True, 2.5, mask)
        return torch.autograd.grad(w.square().sum() + loss + (y * up).sum() + r.sum(), (gain, gate))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(torch.randn(T, H, generator=g))
    mask[50:] = False
    graph.replay()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)
