"""Tokens sorted by expert and back, with gradients, against 64-bit loops.

The order and the copied rows are exact.  Tolerances: an output rounded once to
type u (2^-8 bf16, 2^-24 float32, relative) after a float32 sum of n terms is
within u |ref| + (n + 1) 2^-23 sum|terms| of the exact sum, whatever the order.
"""
import math

import numpy as np
import pytest
import torch

import lora_moe_expert_info_gb300 as mlr
from lora_moe_expert_info_gb300 import permute as pm
from oracle import experts as ox

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def f64(t):
    return t.detach().cpu().double().numpy()


def case(T, K, E, H, dtype, seed=0, masked=0.0, skew=0.0, dev="cuda"):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (T, K))
    if skew:
        ids = np.where(rng.random((T, K)) < skew, E // 2, ids)
    if masked:
        ids = np.where(rng.random((T, K)) < masked, -1, ids)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(dtype).to(dev)
    w = torch.rand(T, K, generator=g).to(dev)
    return x, torch.from_numpy(ids.astype(np.int32)).to(dev), w


SHAPES = [
    # T, K, E, H: one token; sizes off every multiple; rows of 16, 4 and 2 byte vectors; one expert
    (1, 1, 1, 8), (1, 8, 128, 2048), (3, 2, 5, 7), (5, 3, 4, 6), (37, 6, 60, 111), (64, 8, 16, 128), (130, 5, 3, 1001),
    (257, 1, 1, 40), (33, 7, 300, 72),
]


@pytest.mark.parametrize("T,K,E,H", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("masked", [0.0, 0.3, 1.0])
def test_permute_and_back(cuda_device, T, K, E, H, dtype, masked):
    x, ids, w = case(T, K, E, H, dtype, seed=T + K, masked=masked)
    rows, pos, off = pm.moe_permute(x, ids, E)
    rpos, roff = ox.sort_pairs(ids.cpu().numpy(), E)
    assert np.array_equal(pos.cpu().numpy(), rpos) and np.array_equal(off.cpu().numpy(), roff)
    assert np.array_equal(f64(rows), ox.permute(f64(x), rpos))
    pos2, off2 = pm.moe_sort_pairs(ids, E)
    assert torch.equal(pos, pos2) and torch.equal(off, off2)

    r = torch.randn(T * K, H, generator=torch.Generator().manual_seed(5)).to(dtype).to(x.device)
    y = f64(pm.moe_unpermute(r, pos, w, check=True))
    ref, mag = ox.unpermute(f64(r), rpos, f64(w))
    assert np.all(np.abs(y - ref) <= U[dtype] * np.abs(ref) + (K + 1) * 2.0 ** -23 * mag)
    dx = f64(pm.moe_permute_backward(r, pos, check=True))
    ref, mag = ox.unpermute(f64(r), rpos, np.ones((T, K)))
    assert np.all(np.abs(dx - ref) <= U[dtype] * np.abs(ref) + (K + 1) * 2.0 ** -23 * mag)

    dy = x
    d_rows, dw = pm.moe_unpermute_backward(dy, r, pos, w, check=True)
    rd, rw, mag = ox.unpermute_backward(f64(dy), f64(r), rpos, f64(w))
    assert np.all(np.abs(f64(d_rows) - rd) <= (U[dtype] + 2.0 ** -23) * np.abs(rd))
    assert np.all(np.abs(f64(dw) - rw) <= (H + 1) * 2.0 ** -23 * mag)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,K,E,H,masked", [(2000, 8, 60, 72, 0.1), (2000, 8, 60, 71, 0.1), (1500, 6, 7, 4200, 0.05),
                                            (9000, 1, 5, 1, 0.0), (9000, 1, 5, 2, 0.1), (1100, 8, 3, 2083, 0.0),
                                            (50, 2, 3, 5000, 0.2), (50, 3, 3, 4099, 0.2)])
def test_rows_of_large_batches_and_long_rows(cuda_device, T, K, E, H, dtype, masked):
    """Past the single launch, long rows and rows off the 16-byte grid, against
    indexing and 64-bit sums on the device."""
    x, ids, w = case(T, K, E, H, dtype, seed=T + H, masked=masked)
    rows, pos, off = pm.moe_permute(x, ids, E)
    at, held = torch.where(pos < 0, ~pos, pos).long(), pos >= 0
    want = torch.zeros_like(rows)
    want[at.reshape(-1)] = torch.where(held[..., None], x[:, None].expand(-1, K, -1), 0).reshape(T * K, H)
    assert torch.equal(rows, want)
    assert int(off[-1]) == int(held.sum())

    r = torch.randn(T * K, H, generator=torch.Generator().manual_seed(5)).to(dtype).cuda()
    g = torch.where(held[..., None], r[at].double(), 0)
    wd = w.double()[..., None]
    u = U[dtype]

    def near(got, ref, mag, terms):
        return bool(((got.double() - ref).abs() <= u * ref.abs() + (terms + 1) * 2.0 ** -23 * mag).all())

    assert near(pm.moe_unpermute(r, pos, w, check=True), (g * wd).sum(1), (g * wd).abs().sum(1), K)
    assert near(pm.moe_permute_backward(r, pos, check=True), g.sum(1), g.abs().sum(1), K)
    d_rows, dw = pm.moe_unpermute_backward(x, r, pos, w, check=True)
    ref = torch.zeros(T * K, H, dtype=torch.float64, device="cuda")
    ref[at.reshape(-1)] = torch.where(held[..., None], x.double()[:, None] * wd, 0).reshape(T * K, H)
    assert bool(((d_rows.double() - ref).abs() <= (u + 2.0 ** -23) * ref.abs()).all())
    t = g * x.double()[:, None]
    assert bool(((dw.double() - t.sum(-1)).abs() <= (H + 1) * 2.0 ** -23 * t.abs().sum(-1)).all())


@pytest.mark.parametrize("T,K,E,masked,skew", [(1024, 8, 128, 0.0, 0.0), (1025, 8, 128, 0.1, 0.0), (5000, 8, 256, 0.0, 0.9),
                                               (40000, 3, 17, 0.05, 0.0), (9000, 1, 4000, 0.0, 0.0),
                                               (300, 100, 7, 0.2, 0.0), (2, 256, 16384, 0.0, 0.0),
                                               (100, 200, 16384, 0.0, 0.0), (300000, 2, 3, 0.0, 0.0)])
def test_order_of_large_batches(cuda_device, T, K, E, masked, skew):
    """Around and past the largest batch of a single launch, against a stable sort."""
    _, ids, _ = case(T, K, E, 1, F32, seed=E, masked=masked, skew=skew)
    pos, off = pm.moe_sort_pairs(ids, E)
    key = torch.where((ids < 0), E, ids).reshape(-1).long()
    by, order = key.cpu().sort(stable=True)
    want = torch.empty_like(order)
    want[order] = torch.arange(order.numel())
    want = torch.where(key.cpu() < E, want, ~want).int()
    assert torch.equal(pos.cpu().reshape(-1), want)
    assert torch.equal(off.cpu(), torch.searchsorted(by, torch.arange(E + 1)).int())


@pytest.mark.parametrize("T,K,E,masked", [(1025, 8, 128, 0.1), (2048, 8, 60, 0.0), (2049, 8, 60, 0.1), (1366, 12, 16000, 0.1),
                                          (70, 200, 3, 0.0), (16384, 1, 1, 0.5), (16385, 1, 5, 0.0)])
def test_order_with_and_without_rows(cuda_device, T, K, E, masked):
    """Sorting alone takes one launch for larger batches than sorting with rows;
    both orders are the stable sort's."""
    x, ids, _ = case(T, K, E, 8, F32, seed=T, masked=masked)
    rows, pos, off = pm.moe_permute(x, ids, E)
    pos2, off2 = pm.moe_sort_pairs(ids, E)
    assert torch.equal(pos, pos2) and torch.equal(off, off2)
    key = torch.where(ids < 0, E, ids).reshape(-1).long()
    by, order = key.sort(stable=True)
    want = torch.empty_like(order)
    want[order] = torch.arange(order.numel(), device="cuda")
    assert torch.equal(torch.where(pos < 0, ~pos, pos).reshape(-1), want.int())
    assert torch.equal(off, torch.searchsorted(by, torch.arange(E + 1, device="cuda")).int())


def test_no_tokens_and_no_columns(cuda_device):
    x = torch.empty(0, 16, device="cuda", dtype=BF)
    ids = torch.empty(0, 4, device="cuda", dtype=torch.int32)
    rows, pos, off = pm.moe_permute(x, ids, 3)
    assert rows.shape == (0, 16) and pos.shape == (0, 4) and off.tolist() == [0, 0, 0, 0]
    assert pm.moe_permute_backward(rows, pos).shape == (0, 16)
    assert pm.moe_unpermute(rows, pos, torch.empty(0, 4, device="cuda")).shape == (0, 16)
    d_rows, dw = pm.moe_unpermute_backward(x, rows, pos, torch.empty(0, 4, device="cuda"))
    assert d_rows.shape == (0, 16) and dw.shape == (0, 4)
    rows, pos, off = pm.moe_permute(torch.empty(2, 0, device="cuda"), torch.tensor([[1], [0]], device="cuda", dtype=torch.int32), 2)
    assert rows.shape == (2, 0) and pos.tolist() == [[1], [0]] and off.tolist() == [0, 1, 2]


def test_masked_pairs_keep_nan_out(cuda_device):
    """Nothing of a masked pair's weight, row or gradient reaches a result."""
    T, K, E, H = 6, 2, 3, 16
    x, ids, w = case(T, K, E, H, BF, seed=3)
    ids[2, 1] = ids[4, 0] = -1
    rows, pos, off = pm.moe_permute(x, ids, E)
    n = int(off[-1])
    assert n == T * K - 2 and not rows[n:].any()
    rows[n:] = float("nan")
    w[2, 1] = float("inf")
    w[4, 0] = float("nan")
    assert pm.moe_unpermute(rows, pos, w).isfinite().all()
    d_rows, dw = pm.moe_unpermute_backward(x, rows, pos, w)
    assert d_rows.isfinite().all() and not d_rows[n:].any()
    assert dw.isfinite().all() and dw[2, 1] == 0 and dw[4, 0] == 0
    # and those of an unmasked one do
    rows[0] = float("nan")
    assert pm.moe_unpermute(rows, pos, torch.ones_like(w)).isnan().any()


def test_ids_out_of_range_are_masked_and_reported(cuda_device):
    x, ids, _ = case(50, 2, 4, 32, BF, seed=1)
    ids[7, 0], ids[9, 1] = 4, -2
    with pytest.raises(mlr.MoeLoraError) as ei:
        pm.moe_permute(x, ids, 4)
    assert ei.value.code == mlr.MLR_ERR_INDEX
    rows, pos, off = pm.moe_permute(x, ids, 4, check=False)
    want = ids.cpu().numpy().copy()
    want[7, 0] = want[9, 1] = -1
    rpos, roff = ox.sort_pairs(want, 4)
    assert np.array_equal(pos.cpu().numpy(), rpos) and np.array_equal(off.cpu().numpy(), roff)
    ids[7, 0] = ids[9, 1] = -1
    pm.moe_permute(x, ids, 4)  # -1 masks silently


def test_places_out_of_range_are_reported(cuda_device):
    x, ids, w = case(8, 2, 4, 32, F32, seed=1)
    rows, pos, _ = pm.moe_permute(x, ids, 4)
    pos[3, 1] = 16
    pos[5, 0] = ~16
    for call in (lambda: pm.moe_unpermute(rows, pos, w, check=True),
                 lambda: pm.moe_unpermute_backward(x, rows, pos, w, check=True)):
        with pytest.raises(mlr.MoeLoraError) as ei:
            call()
        assert ei.value.code == mlr.MLR_ERR_INDEX


def test_unaligned_views(cuda_device):
    """Contiguous tensors that begin off a 16-byte boundary take narrower vectors."""
    T, K, E, H = 20, 3, 4, 64
    x, ids, w = case(T, K, E, H, BF, seed=2)
    base = torch.empty(T * H + 1, device="cuda", dtype=BF)
    xu = base[1:].view(T, H)
    xu.copy_(x)
    rows, pos, _ = pm.moe_permute(x, ids, E)
    rows2, _, _ = pm.moe_permute(xu, ids, E)
    assert torch.equal(rows, rows2)
    rb = torch.empty(T * K * H + 2, device="cuda", dtype=BF)
    ru = rb[2:].view(T * K, H)
    ru.copy_(rows)
    assert torch.equal(pm.moe_unpermute(rows, pos, w), pm.moe_unpermute(ru, pos, w))
    a, b = pm.moe_unpermute_backward(x, rows, pos, w), pm.moe_unpermute_backward(xu, ru, pos, w)
    assert torch.equal(a[0], b[0])
    assert torch.allclose(a[1], b[1], rtol=1e-5, atol=(H + 1) * 2.0 ** -23 * H)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,K,E,H", [(3, 2, 4, 1), (70, 3, 5, 3), (9, 4, 3, 8), (600, 2, 7, 64), (300, 3, 9, 256),
                                     (21, 5, 6, 1111), (5, 2, 3, 1024), (1100, 8, 20, 37)])
def test_copies_at_any_address(cuda_device, dtype, T, K, E, H):
    """x and rows at every address their type allows, NaN around both: the rows
    are those at 512-byte boundaries, nothing around x is read into them and
    nothing around rows is written."""
    x, ids, _ = case(T, K, E, H, dtype, seed=H, masked=0.1)
    want, pos, off = pm.moe_permute(x, ids, E)

    def at(shape, k):  # a view k elements past a boundary, NaN around it
        n = math.prod(shape)
        buf = torch.full((n + 32,), math.nan, dtype=dtype, device="cuda")
        return buf, buf[k:k + n].view(shape)

    per = 16 // x.element_size()
    for k in range(per + 1):
        for j in range(per):
            _, xk = at(x.shape, k)
            xk.copy_(x)
            buf, rows = at(want.shape, j)
            pm.moe_permute(xk, ids, E, rows=rows)
            assert torch.equal(rows, want)
            assert buf[:j].isnan().all() and buf[j + rows.numel():].isnan().all()


def test_buffers_streams_and_repeats(cuda_device):
    T, K, E, H = 700, 8, 32, 256
    x, ids, w = case(T, K, E, H, BF, seed=4, masked=0.1)
    rows, pos, off = pm.moe_permute(x, ids, E)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    rows2 = torch.full_like(rows, 7)
    out = pm.moe_permute(x, ids, E, rows=rows2, stream=s, check=False)
    y2 = pm.moe_unpermute(rows2, out[1], w, stream=s)
    g2 = pm.moe_unpermute_backward(x, rows2, out[1], w, stream=s)
    s.synchronize()
    assert out[0] is rows2 and torch.equal(rows, rows2) and torch.equal(pos, out[1]) and torch.equal(off, out[2])
    assert torch.equal(pm.moe_unpermute(rows, pos, w), y2)
    g = pm.moe_unpermute_backward(x, rows, pos, w)
    assert torch.equal(g[0], g2[0]) and torch.equal(g[1], g2[1])


def test_rows_past_32_bit_offsets(cuda_device):
    """Rows whose element offsets pass 2^31 and byte offsets 2^32."""
    T, K, E, H = 40000, 8, 4, 7168
    ids = (torch.arange(T * K, device="cuda", dtype=torch.int32).reshape(T, K) * 7) % E
    x = torch.randn(T, H, device="cuda", dtype=BF)
    rows, pos, _ = pm.moe_permute(x, ids, E)
    assert rows.numel() > 2 ** 31
    last = rows[-3:].clone()
    order = pos.reshape(-1).long().argsort()
    assert torch.equal(last, x[order[-3:] // K])
    y = pm.moe_unpermute(rows, pos, torch.full((T, K), 0.125, device="cuda"))
    assert torch.equal(y, x)  # eight equal rows weighted by an eighth
    d_rows, dw = pm.moe_unpermute_backward(x, rows, pos, torch.full((T, K), 2.0, device="cuda"))
    assert torch.equal(d_rows[-3:], 2 * last)
    assert torch.allclose(dw[-1], (x[-1].float() ** 2).sum().expand(K), rtol=1e-4)


def test_gradients_against_differences(cuda_device):
    """A loss through permute, a per-row scaling and unpermute: autograd's
    directional derivative against a central difference of the loss taken in 64
    bits.  The loss is a polynomial of degree 2 in x and 1 in w along the
    direction, so the difference is exact up to rounding; float32 gradients of
    about N products carry a relative error of at most N 2^-23."""
    T, K, E, H = 12, 3, 4, 24
    x, ids, w = case(T, K, E, H, F32, seed=8, masked=0.1)
    gain = torch.linspace(0.5, 1.5, T * K, device="cuda")[:, None]
    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    rows, pos, _ = pm.MoePermute.apply(xr, ids, E)
    y = pm.MoeUnpermute.apply(rows * gain, pos, wr)
    (0.5 * y.square()).sum().backward()
    p = pos.cpu().numpy()

    def loss(x64, w64):
        r = ox.permute(x64, p) * gain.cpu().double().numpy()
        return 0.5 * (ox.unpermute(r, p, w64)[0] ** 2).sum()

    rng = np.random.default_rng(0)
    vx, vw = rng.standard_normal((T, H)), rng.standard_normal((T, K))
    h = 1e-4
    for dx_, dw_, grad in ((vx, 0 * vw, (f64(xr.grad) * vx).sum()), (0 * vx, vw, (f64(wr.grad) * vw).sum())):
        num = (loss(f64(x) + h * dx_, f64(w) + h * dw_) - loss(f64(x) - h * dx_, f64(w) - h * dw_)) / (2 * h)
        size = np.abs(f64(xr.grad) * vx).sum() + np.abs(f64(wr.grad) * vw).sum()
        assert abs(num - grad) <= (T * K * H) * 2.0 ** -23 * size + 1e-6 * abs(num)


def test_graph_replay(cuda_device):
    """No call decides anything on the host from device data: a captured step
    replays on new inputs."""
    T, K, E, H = 300, 4, 16, 128
    x, ids, w = case(T, K, E, H, BF, seed=1)
    ws = torch.empty(pm._lib().moe_permute_workspace_bytes(T, K, E), dtype=torch.uint8, device="cuda")
    rows = torch.empty(T * K, H, dtype=BF, device="cuda")
    pos = torch.empty(T, K, dtype=torch.int32, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    y = torch.empty(T, H, dtype=BF, device="cuda")

    def step():
        pm.moe_permute(x, ids, E, rows=rows, pair_pos=pos, expert_offsets=off, workspace=ws, check=False)
        pm.moe_unpermute(rows, pos, w, y=y)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step()
    x2, ids2, w2 = case(T, K, E, H, BF, seed=9, masked=0.2)
    x.copy_(x2), ids.copy_(ids2), w.copy_(w2)
    g.replay()
    torch.cuda.synchronize()
    r2, p2, o2 = pm.moe_permute(x2, ids2, E)
    assert torch.equal(rows, r2) and torch.equal(pos, p2) and torch.equal(off, o2)
    assert torch.equal(y, pm.moe_unpermute(r2, p2, w2))
