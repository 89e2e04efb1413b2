"""The router's choice, the balance loss and their gradients against 64 bits.

Ids are exact.  Tolerances: exp of a rounded difference d of logits is within
(|d| + 4) 2^-24 of exact; sums of E positive terms within E 2^-24; so for |d| < 40 a
weight is within (E + 64) 2^-23 of itself (one more factor of two for quotients), a
gradient within as much of the magnitude of its terms, then rounded once to its type
(half a step: bf16 2^-8, float32 2^-24).
"""
import math

import numpy as np
import pytest
import torch

import lora_moe_expert_info_gb300 as mlr
from lora_moe_expert_info_gb300 import permute as pm, router as rt
from oracle import router as ox

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def f64(t):
    return t.detach().cpu().double().numpy()


def logits_of(T, E, dtype=F32, seed=0, closed=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) + 0.5 * torch.randn(E, generator=g)
    if closed:
        l[:, torch.randperm(E, generator=g)[:closed]] = -math.inf
    out = torch.empty(T * E + shift, dtype=dtype, device="cuda")[shift:].view(T, E)
    return out.copy_(l.to(dtype))


def check_route(l, K, scoring="softmax", bias=None, groups=1, best=1, renormalize=True, scale=1.0, mask=None):
    E = l.shape[1]
    ids, w = rt.moe_route(l, K, scoring, bias, groups, best, renormalize, scale, mask)
    m = None if mask is None else mask.cpu().numpy()
    ref = ox.choose(f64(l), K, scoring, None if bias is None else f64(bias), groups, best, m)
    assert np.array_equal(ids.cpu().numpy(), ref)
    rw = ox.weights(f64(l), ref, scoring, renormalize, scale)
    assert np.all(np.abs(f64(w) - rw) <= (E + 64) * 2.0 ** -23 * np.abs(rw) + 2.0 ** -140)
    return ids, w, ref


SHAPES = [(1, 1, 1), (1, 128, 8), (3, 2, 1), (5, 7, 3), (40, 16, 16), (33, 31, 2), (70, 60, 6), (9, 65, 32), (257, 128, 8), (6, 100, 10),
          (130, 256, 8), (50, 256, 1), (4, 384, 8), (12, 512, 10), (3, 1000, 8), (2, 1024, 32), (2, 4096, 16), (3, 4001, 4)]


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route(cuda_device, T, E, K, dtype, scoring, renormalize):
    for shift in (0, 1):
        l = logits_of(T, E, dtype, seed=T + E, shift=shift)
        check_route(l, K, scoring, renormalize=renormalize, scale=2.5)
    if scoring == "sigmoid":
        bias = 0.05 * torch.randn(E, generator=torch.Generator().manual_seed(1)).cuda()
        check_route(l, K, scoring, bias, renormalize=renormalize)
    if T > 1 and E > 8:
        mask = torch.arange(T, device="cuda") % 3 != 1
        l = logits_of(T, E, dtype, seed=9, closed=E // 8)
        l[1::3] = math.nan  # padding holds anything
        ids, w, _ = check_route(l, K, scoring, renormalize=renormalize, mask=mask)
        assert (ids[1::3] == -1).all() and not w[1::3].any()
        rt.moe_route(l, K, scoring, token_mask=mask, check=True)  # what is masked is not looked at


@pytest.mark.parametrize("E,G,best,K", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 2, 1, 6), (60, 4, 2, 6), (8, 8, 3, 3), (24, 12, 5, 8), (512, 8, 8, 10),
                                        (33, 11, 4, 5), (1024, 256, 30, 32), (256, 4, 2, 12), (96, 32, 2, 4)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_groups(cuda_device, E, G, best, K, scoring, with_bias, dtype):
    bias = 0.05 * torch.randn(E, generator=torch.Generator().manual_seed(1)).cuda() if with_bias and scoring == "sigmoid" else None
    check_route(logits_of(130, E, dtype, seed=E), K, scoring, bias, G, best, scale=2.5)
    check_route(logits_of(40, E, dtype, seed=E + 1, closed=E // 2), K, scoring, bias, G, best, renormalize=False)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K,G,best", [(256, 8, 1, 1), (256, 8, 8, 4), (60, 6, 1, 1), (60, 6, 4, 2), (512, 10, 1, 1), (4000, 8, 1, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_ties_go_to_the_lowest_index(cuda_device, scoring, E, K, G, best, dtype):
    l = torch.zeros(6, E, dtype=dtype, device="cuda")
    l[1] = 3.0e38
    l[2] = -3.0e38  # a mask of the type's lowest value is a logit like any other
    l[3, E // 2:] = 1.0
    l[4, ::2] = 0.5
    l[5] = -0.0
    l[5, 1::2] = 0.0  # the zeros are equal
    bias = torch.full((E,), 0.25, device="cuda") if scoring == "sigmoid" else None
    ids, w, _ = check_route(l, K, scoring, bias, G, best)
    if G == 1:
        assert ids[0].tolist() == ids[5].tolist() == list(range(K))
    # coarse logits: ties everywhere
    l = (logits_of(200, E, F32, seed=3) * 2).round().to(dtype) / 2
    check_route(l, K, scoring, bias, G, best)
    if scoring == "sigmoid":
        check_route(l, K, scoring, None, G, best)
        check_route(l, K, scoring, (bias * 40).round() / 40, G, best)


@pytest.mark.parametrize("E,K", [(64, 8), (128, 1), (130, 16), (256, 8), (256, 10), (392, 8), (512, 16), (1000, 6), (1024, 12)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift", [0, 1])
def test_rows_of_equal_logits(cuda_device, E, K, dtype, shift):
    """Rows of one value, with none to many logits above it, and others below."""
    T = 90
    rng = np.random.default_rng(E + K)
    rows = np.zeros((T, E))
    for t in range(T):
        rows[t] = rng.choice([0.0, -0.0, 1.5, -3.25])
        at = rng.permutation(E)
        more = (0, 1, K - 1, K, K + 3, 30, 31, 32, 40, E // 2)[t % 10]
        rows[t, at[:more]] = 4 + rng.integers(0, 1 + t % 3, more)
        rows[t, at[more:more + (t % 4) * E // 8]] = -8.0
    l = torch.empty(T * E + shift, dtype=dtype, device="cuda")[shift:].view(T, E)
    l.copy_(torch.from_numpy(rows))
    check_route(l, K)
    check_route(l, K, "sigmoid", renormalize=False)
    if E % 8 == 0:
        check_route(l, min(K, E // 4), "softmax", None, 8, 2, renormalize=False)


@pytest.mark.parametrize("E,G,best,K", [(64, 1, 1, 8), (256, 1, 1, 8), (256, 8, 4, 8), (256, 8, 2, 16), (520, 1, 1, 10), (96, 8, 3, 6), (1000, 4, 1, 6)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_equal_scores(cuda_device, E, G, best, K, dtype):
    """The same for sigmoid scoring: biases of one value, of a few, and of values that
    32 bits hardly tell apart, over rows of a few logits."""
    T = 80
    rng = np.random.default_rng(E + G)
    l = np.zeros((T, E))
    for t in range(T):
        l[t] = rng.choice([0.0, 1.5, -2.0])
        at = rng.permutation(E)
        more = (0, 1, K, 31, 40, E // 2)[t % 6]
        l[t, at[:more]] = 0.25 * rng.integers(-8, 9, more)
    l = torch.from_numpy(l).to(dtype).cuda()
    steps = torch.from_numpy(rng.integers(0, 3, E)).cuda()
    for bias in (None, torch.zeros(E, device="cuda"), 0.5 * steps.float(), 0.3 + steps.float() * 2.0 ** -24,
                 torch.where(steps == 0, 0.7, 0.3).float()):
        check_route(l, K, "sigmoid", bias, G, best)


def test_biases_whose_sums_pass_the_range(cuda_device):
    """Scores near float32's largest, whose pairs' sums are beyond it, still have an order."""
    E, G = 32, 4
    bias = torch.zeros(E, device="cuda")
    for i, b in {1: 2.0e38, 5: 3.0e38, 8: 3.1e38, 9: 2.5e38, 20: 3.3e38, 22: 3.0e38, 27: 1.0e38, -1: 2.0e37}.items():
        bias[i] = b
    l = logits_of(64, E, seed=5)
    for best in (1, 2, 3):
        check_route(l, 4, "sigmoid", bias, G, best)
        check_route(l, 4, "sigmoid", -bias, G, best)


@pytest.mark.parametrize("E,G,best", [(64, 1, 1), (256, 1, 1), (64, 4, 2), (256, 8, 4)])
def test_scores_that_32_bits_do_not_tell_apart(cuda_device, E, G, best):
    """Pairs of experts whose sigmoid + bias differ by about 1e-8, in either order."""
    T = 300
    rng = np.random.default_rng(E)
    bias = (0.3 * rng.random(E)).astype(np.float32)
    l = rng.normal(size=(T, E)).astype(np.float32)
    for i in range(0, E - 1, 2):
        want = ox.sigmoid(l[:, i].astype(float)) + float(bias[i]) - float(bias[i + 1])
        ok = (want > 0.01) & (want < 0.99)
        with np.errstate(invalid="ignore", divide="ignore"):
            l[:, i + 1] = np.where(ok, np.log(want / (1 - want)), l[:, i + 1])
    c = ox.sigmoid(l.astype(float)) + bias
    gap = np.abs(c[:, ::2] - c[:, 1::2])
    assert np.median(gap) < 3e-8 and (gap > 1e-12).mean() > 0.9  # the case is what it says
    lt, bt = torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda()
    for K in (1, 4, 7, 8):
        check_route(lt, K, "sigmoid", bt, G, best)
    # a bias so large that 32-bit sums lose the sigmoids' last bits
    check_route(lt, 8, "sigmoid", bt + 1000, G, best)


def test_groups_that_32_bits_do_not_tell_apart(cuda_device):
    """Two groups of the same pair of experts, one of them a step apart in float32."""
    E, G = 32, 4
    rng = np.random.default_rng(0)
    l = rng.normal(size=(200, E)).astype(np.float32) - 4
    top = rng.normal(size=(200, 2)).astype(np.float32)
    for g in range(G):
        l[:, 8 * g + 1], l[:, 8 * g + 6] = top[:, 0], top[:, 1]
    flip = rng.integers(0, G, 200)
    at = np.arange(200), 8 * flip + 6
    l[at] = np.nextafter(l[at], np.where(rng.random(200) < 0.5, -9, 9).astype(np.float32))
    for best in (1, 2, 3):
        check_route(torch.from_numpy(l).cuda(), 4, "sigmoid", None, G, best)
        check_route(torch.from_numpy(l).cuda(), 4, "sigmoid", torch.full((E,), 0.5, device="cuda"), G, best)


def test_closed_experts_and_empty_rows(cuda_device):
    E, K = 16, 4
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            l = logits_of(7, E, seed=2)
            l[0] = -math.inf
            l[1, 2:] = -math.inf
            l[2, 1:] = math.nan
            l[3, 5] = math.inf
            l[4] = math.nan
            ids, w, _ = check_route(l, K, scoring, renormalize=renormalize)
            assert (ids[0] == -1).all() and not w[0].any() and (ids[1] >= 0).sum() == 2 and torch.isfinite(w).all()
            g = torch.randn(7, K, device="cuda")
            d = rt.moe_route_backward(l, ids, g, scoring=scoring, renormalize=renormalize)
            assert torch.isfinite(d).all() and not d[0].any() and not d[4].any() and not d[1, 2:].any()
            with pytest.raises(mlr.MoeLoraError, match="NaN"):
                rt.moe_route(l, K, scoring, renormalize=renormalize, check=True)
            rt.moe_route(l[:2], K, scoring, renormalize=renormalize, check=True)  # -inf closes an expert silently
            loss, counts = rt.moe_balance_loss(l, ids, scoring)
            ref, rc = ox.balance(f64(l), ids.cpu().numpy(), scoring)
            assert abs(float(loss) - ref) <= 100 * 2.0 ** -23 * ref and np.array_equal(counts.cpu().numpy(), rc)
    # biases that close experts
    bias = torch.zeros(E, device="cuda")
    bias[3], bias[4], bias[5] = -math.inf, math.nan, math.inf
    l = logits_of(5, E, seed=4)
    l[:, 3:6] += 5
    ids, _ = rt.moe_route(l, K, "sigmoid", bias)
    ref = ox.choose(f64(l), K, "sigmoid", f64(bias))
    assert np.array_equal(ids.cpu().numpy(), ref) and not np.isin(ref, [3, 4, 5]).any()
    # sigmoids that are all zero have no shares
    ids, w = rt.moe_route(torch.full((2, E), -3.0e38, device="cuda"), K, "sigmoid")
    assert ids.tolist() == [[0, 1, 2, 3]] * 2 and not w.any()
    d = rt.moe_route_backward(torch.full((2, E), -3.0e38, device="cuda"), ids, torch.ones(2, K, device="cuda"), scoring="sigmoid")
    assert not d.any()


@pytest.mark.parametrize("T,E,K", SHAPES + [(2000, 64, 4), (3000, 256, 8), (700, 900, 4)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("padded", [False, True])
def test_loss_and_gradients(cuda_device, T, E, K, dtype, scoring, padded):
    l = logits_of(T, E, dtype, seed=E, closed=E // 9)
    mask = (torch.arange(T, device="cuda") % 4 != 2) if padded else None
    m = None if mask is None else mask.cpu().numpy()
    if padded:
        l[2::4] = math.nan
    ids, _ = rt.moe_route(l, K, scoring, token_mask=mask)
    ids_n, ln = ids.cpu().numpy(), f64(l)
    loss, counts = rt.moe_balance_loss(l, ids, scoring, mask)
    ref, rc = ox.balance(ln, ids_n, scoring, m)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert abs(float(loss) - ref) <= (T + E + 64) * 2.0 ** -23 * ref
    assert loss.shape == () and torch.equal(rt.moe_balance_loss(l, ids, scoring, mask)[0], loss)
    d_loss = torch.tensor([0.3], device="cuda")
    rb = ox.balance_backward(float(d_loss), ln, rc, K, scoring, m)
    most = 2 * float(d_loss) * rc[:E].max() * E / (K * max(int(rc[E]), 1) ** 2)
    eps = (E + K + 64) * 2.0 ** -23
    d = rt.moe_route_backward(l, ids, counts=counts, d_loss=d_loss, scoring=scoring, token_mask=mask)
    assert np.all(np.abs(f64(d) - rb) <= U[dtype] * np.abs(rb) + eps * most)
    g = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).cuda()
    for renormalize in (True, False):
        rw = ox.weights_backward(f64(g), ln, ids_n, scoring, renormalize, 2.5)
        mag = 5 * np.abs(f64(g)).sum(1, keepdims=True)
        dw = rt.moe_route_backward(l, ids, g, scoring=scoring, renormalize=renormalize, scale=2.5, token_mask=mask)
        assert np.all(np.abs(f64(dw) - rw) <= U[dtype] * np.abs(rw) + eps * mag)
        if not padded:  # masked tokens have no ids, so the mask need not be given
            assert torch.equal(rt.moe_route_backward(l, ids, g, scoring=scoring, renormalize=renormalize, scale=2.5), dw)
        both = rt.moe_route_backward(l, ids, g, counts, d_loss, scoring, renormalize, 2.5, mask, check=True)
        assert np.all(np.abs(f64(both) - rw - rb) <= U[dtype] * np.abs(rw + rb) + eps * (mag + most))


def test_masked_tokens_without_the_mask(cuda_device):
    """ids of -1 alone: no gradient by the weights."""
    l = logits_of(30, 64)
    mask = torch.arange(30, device="cuda") < 20
    ids, _ = rt.moe_route(l, 4, token_mask=mask)
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            d = rt.moe_route_backward(l, ids, torch.ones(30, 4, device="cuda"), scoring=scoring, renormalize=renormalize)
            assert not d[20:].any() and torch.isfinite(d).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("E", [12, 700])
def test_the_same_expert_twice(cuda_device, scoring, renormalize, E):
    l = logits_of(50, E)
    ids = torch.randint(-1, 4, (50, 6), generator=torch.Generator().manual_seed(0)).int().cuda()
    g = torch.randn(50, 6, generator=torch.Generator().manual_seed(1)).cuda()
    d = rt.moe_route_backward(l, ids, g, scoring=scoring, renormalize=renormalize, check=True)
    ref = ox.weights_backward(f64(g), f64(l), ids.cpu().numpy(), scoring, renormalize, 1.0)
    assert np.all(np.abs(f64(d) - ref) <= (E + 70) * 2.0 ** -23 * 2 * np.abs(f64(g)).sum(1, keepdims=True))
    assert torch.equal(d, rt.moe_route_backward(l, ids, g, scoring=scoring, renormalize=renormalize))


def test_ids_out_of_range(cuda_device):
    l = logits_of(10, 8)
    ids = torch.zeros(10, 2, dtype=torch.int32, device="cuda")
    ids[3, 1], ids[4, 0] = 8, -2
    fine = ids.clone()
    fine[3, 1] = fine[4, 0] = -1
    g = torch.ones(10, 2, device="cuda")
    loss, counts = rt.moe_balance_loss(l, ids)
    assert int(counts[:-1].sum()) == 18 and torch.equal(loss, rt.moe_balance_loss(l, fine, check=True)[0])
    d = rt.moe_route_backward(l, ids, g)
    assert torch.equal(d, rt.moe_route_backward(l, fine, g, check=True))
    for bad in (lambda: rt.moe_balance_loss(l, ids, check=True), lambda: rt.moe_route_backward(l, ids, g, check=True)):
        with pytest.raises(mlr.MoeLoraError) as e:
            bad()
        assert e.value.code == mlr.MLR_ERR_INDEX


def test_empty_batch(cuda_device):
    l = torch.empty(0, 32, device="cuda")
    ids, w = rt.moe_route(l, 4, check=True)
    assert ids.shape == w.shape == (0, 4)
    loss, counts = rt.moe_balance_loss(l, ids)
    assert float(loss) == 0 and counts.tolist() == [0] * 33
    assert rt.moe_route_backward(l, ids, w).shape == (0, 32)
    l = logits_of(5, 32)  # a batch of nothing but padding
    mask = torch.zeros(5, dtype=torch.bool, device="cuda")
    ids, w = rt.moe_route(l, 4, token_mask=mask)
    loss, counts = rt.moe_balance_loss(l, ids, token_mask=mask)
    assert float(loss) == 0 and not counts.any() and (ids == -1).all()
    d = rt.moe_route_backward(l, ids, w, counts, torch.ones(1, device="cuda"), token_mask=mask)
    assert not d.any()


def test_buffers_are_written_in_place(cuda_device):
    l = logits_of(20, 64)
    ids, w = torch.full((30, 4), 77, dtype=torch.int32, device="cuda"), torch.full((30, 4), 7.0, device="cuda")
    a, b = rt.moe_route(l, 4, topk_ids=ids[:20], topk_weights=w[:20])
    assert a.data_ptr() == ids.data_ptr() and (ids[20:] == 77).all() and (w[20:] == 7).all()
    d = torch.full((30, 64), 5.0, device="cuda")
    rt.moe_route_backward(l, a, b, d_logits=d[:20])
    assert (d[20:] == 5).all() and not (d[:20] == 5).any()
    counts, loss = torch.full((66,), 9, dtype=torch.int32, device="cuda"), torch.full((), 9.0, device="cuda")
    assert rt.moe_balance_loss(l, a, loss=loss, counts=counts[:65])[0] is loss and int(counts[65]) == 9
    with pytest.raises(ValueError):
        rt.moe_route(l, 4, topk_ids=ids)


def test_differences(cuda_device):
    """MoeRoute's gradients against differences of its own outputs."""
    for scoring, kw in (("softmax", (None, 1, 1, True, 1.0)), ("softmax", (None, 4, 2, False, 2.0)),
                        ("sigmoid", (torch.linspace(0, 0.1, 16).cuda(), 4, 2, True, 2.5)), ("sigmoid", (None, 1, 1, False, 1.0))):
        l = logits_of(6, 16, seed=11).requires_grad_()
        up = torch.randn(6, 3, generator=torch.Generator().manual_seed(2)).cuda()
        w, ids, loss, counts = rt.MoeRoute.apply(l, 3, scoring, *kw)
        (w * up).sum().add(loss * 3).backward()
        base, idn, upn = f64(l), ids.cpu().numpy(), f64(up)

        def value(v):
            p = ox.scores(v, scoring)
            p = p / p.sum(1, keepdims=True)
            part = (p.sum(0) * counts[:-1].cpu().numpy()).sum() * 16 / (3 * 36)
            return (ox.weights(v, idn, scoring, kw[3], kw[4]) * upn).sum() + 3 * part
        for i in range(6):
            for j in range(0, 16, 3):
                h = np.zeros_like(base)
                h[i, j] = 1e-5
                want = (value(base + h) - value(base - h)) / 2e-5
                assert abs(float(l.grad[i, j]) - want) < 1e-4
        l2 = l.detach().clone().requires_grad_()
        rt.MoeRoute.apply(l2, 3, scoring, *kw)[0].mul(up).sum().backward()
        l3 = l.detach().clone().requires_grad_()
        (rt.MoeRoute.apply(l3, 3, scoring, *kw)[2] * 3).backward()
        assert torch.allclose(l2.grad + l3.grad, l.grad, atol=1e-5)


def test_graphs_and_streams(cuda_device):
    """Two captured graphs of the same calls, replayed on new inputs one after the
    other and on streams of their own, against eager calls."""
    sets = [(logits_of(500, 256, seed=i), torch.randn(500, 8, device="cuda")) for i in range(2)]
    bias, one = 0.05 * torch.randn(256, device="cuda"), torch.ones(1, device="cuda")

    def call(l, g):
        ids, w = rt.moe_route(l, 8, "sigmoid", bias, 8, 4, True, 2.5)
        loss, counts = rt.moe_balance_loss(l, ids, "sigmoid")
        return ids, w, loss, counts, rt.moe_route_backward(l, ids, g, counts, one, "sigmoid", True, 2.5)

    call(*sets[0])
    graphs, got = [], []
    for s in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(call(*s))
    for i, (l, g) in enumerate(sets):
        l.copy_(logits_of(500, 256, seed=20 + i))
    torch.cuda.synchronize()
    for graph in graphs:
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for s, out in zip(sets, got):
        for a, b in zip(call(*s), out):
            assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    l = sets[0][0]
    ids, w = rt.moe_route(l, 8, "sigmoid", bias, 8, 4, True, 2.5, stream=side)
    loss, counts = rt.moe_balance_loss(l, ids, "sigmoid", stream=side)
    d = rt.moe_route_backward(l, ids, sets[0][1], counts, one, "sigmoid", True, 2.5, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((ids, w, loss, counts, d), got[0]):
        assert torch.equal(a, b)


def test_offsets_beyond_32_bits(cuda_device):
    T, E, K = (1 << 21) + 5, 1032, 4
    l = torch.zeros(T, E, dtype=BF, device="cuda")
    tail = logits_of(7, E, BF, seed=1)
    l[-7:] = tail
    ids, w = rt.moe_route(l, K)
    i2, w2 = rt.moe_route(tail, K)
    assert torch.equal(ids[-7:], i2) and torch.equal(w[-7:], w2) and (ids[:-7] == torch.arange(K, device="cuda")).all()
    d = rt.moe_route_backward(l, ids, w)
    assert torch.equal(d[-7:], rt.moe_route_backward(tail, i2, w2))
    loss, counts = rt.moe_balance_loss(l, ids)
    assert int(counts[-1]) == T and int(counts[:-1].sum()) == T * K and abs(float(loss) - 1) < 1e-2


def test_choice_feeds_the_sort(cuda_device):
    """Ids of padded tokens are masked pairs of the sort, the counts its offsets."""
    l = logits_of(100, 32, closed=5)
    mask = torch.arange(100, device="cuda") < 90
    ids, w = rt.moe_route(l, 4, token_mask=mask)
    _, counts = rt.moe_balance_loss(l, ids, token_mask=mask)
    _, offsets = pm.moe_sort_pairs(ids, 32)
    assert torch.equal(offsets[1:] - offsets[:-1], counts[:-1]) and int(offsets[-1]) == 90 * 4
