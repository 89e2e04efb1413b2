"""The norm, its 8 bits and its gradients against 64 bits.

Tolerances.  With u half a step of the output's type (bf16 2^-8, float32 2^-24)
and H positive terms summed in float32, whatever the order: the sum is within
H 2^-24 of the exact one, its root's inverse within half of that and the few
roundings around it, so y is within (u + (H / 2 + 8) 2^-24) |y|.  Gradients are sums whose
terms have the magnitude `mag`, each within (H + 16) 2^-24 of itself (m^3's error
is 3 H / 2 2^-24, the dot product's H 2^-24: 3 H in all), then rounded once.
"""
import math

import numpy as np
import pytest
import torch

from lora_moe_expert_info_gb300 import norm
from oracle import router as ox

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def f64(t):
    return t.detach().cpu().double().numpy()


def make(T, H, dtype, w_dtype=None, seed=0, shift=0):
    """x, residual, weight; with a shift, rows that begin so many elements after a 16-byte boundary."""
    g = torch.Generator().manual_seed(seed)

    def rows(scale):
        v = (torch.randn(T * H, generator=g) * scale).to(dtype)
        out = torch.empty(T * H + shift, dtype=dtype, device="cuda")[shift:].view(T, H)
        return out.copy_(v.view(T, H))

    return rows(1.0), rows(3.0), (1 + 0.2 * torch.randn(H, generator=g)).to(w_dtype or dtype).cuda()


# rows of one column, below a vector, of 16-byte vectors and off them, ending inside a
# group of 128 and at its end, one and several to a block, up to the largest
SHAPES = [(1, 1), (3, 7), (5, 8), (33, 128), (7, 129), (9, 200), (4, 256), (130, 1000), (3, 1111), (2, 2048), (17, 2056), (5, 4099),
          (2, 7168), (3, 8200), (3, 8203), (2, 12288), (1, 16381), (2, 16384)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift", [0, 1])
def test_forward(cuda_device, T, H, dtype, shift):
    x, res, w = make(T, H, dtype, seed=T + H, shift=shift)
    y, r = norm.rms_norm(x, w, 1e-6)
    assert r is x
    ref = ox.norm(f64(x), f64(w), 1e-6)
    assert np.all(np.abs(f64(y) - ref) <= (U[dtype] + (H / 2 + 8) * 2.0 ** -24) * np.abs(ref))
    y, r = norm.rms_norm(x, w, 1e-6, res)
    total = f64(x) + f64(res)
    assert np.all(np.abs(f64(r) - total) <= (U[dtype] + 2.0 ** -24) * np.abs(total))
    assert torch.equal(r, (x.float() + res.float()).to(dtype))
    ref = ox.norm(f64(r), f64(w), 1e-6)
    assert np.all(np.abs(f64(y) - ref) <= (U[dtype] + (H / 2 + 8) * 2.0 ** -24) * np.abs(ref))
    codes, exps, y8, r8 = norm.rms_norm_fp8(x, w, 1e-6, res)
    assert torch.equal(y8, y) and torch.equal(r8, r)
    rc, re = ox.eight_bits(f64(y))
    assert np.array_equal(exps.cpu().numpy(), re) and np.array_equal(codes.cpu().numpy(), rc)
    c2, e2, none, _ = norm.rms_norm_fp8(x, w, 1e-6, res, with_y=False)
    assert none is None and torch.equal(c2, codes) and torch.equal(e2, exps)
    back = ox.from_eight_bits(rc, re)
    for out in (BF, F32):
        assert np.array_equal(f64(norm.fp8_dequantize(codes, exps, out)), back)


@pytest.mark.parametrize("T,H", SHAPES + [(700, 96), (1300, 2048), (650, 1111)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shift", [0, 3])
def test_gradients(cuda_device, T, H, dtype, shift):
    r, dy, w = make(T, H, dtype, seed=T * H, shift=shift)
    d_r = make(T, H, dtype, seed=5, shift=shift)[0]
    for e in (None, d_r):
        dx, dw = norm.rms_norm_backward(dy, r, w, 1e-5, e)
        rx, rw, mx, mw = ox.norm_backward(f64(dy), f64(r), f64(w), 1e-5, None if e is None else f64(e))
        assert np.all(np.abs(f64(dx) - rx) <= U[dtype] * np.abs(rx) + (3 * H + 16) * 2.0 ** -24 * mx)
        assert np.all(np.abs(f64(dw) - rw) <= (H + T + 16) * 2.0 ** -24 * mw)
        again = norm.rms_norm_backward(dy, r, w, 1e-5, e)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dtype,w_dtype", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("H", [256, 777])
def test_weight_of_the_other_type(cuda_device, dtype, w_dtype, H):
    x, res, w = make(40, H, dtype, w_dtype)
    y, r = norm.rms_norm(x, w, 1e-6, res)
    ref = ox.norm(f64(r), f64(w), 1e-6)
    assert np.all(np.abs(f64(y) - ref) <= (U[dtype] + (H / 2 + 8) * 2.0 ** -24) * np.abs(ref))
    dx, dw = norm.rms_norm_backward(x, r, w, 1e-6)
    rx, rw, mx, mw = ox.norm_backward(f64(x), f64(r), f64(w), 1e-6)
    assert np.all(np.abs(f64(dx) - rx) <= U[dtype] * np.abs(rx) + (3 * H + 16) * 2.0 ** -24 * mx)
    assert np.all(np.abs(f64(dw) - rw) <= (H + 56) * 2.0 ** -24 * mw)


def test_extreme_rows(cuda_device):
    """Zero rows, groups of zeros, the largest and smallest numbers, infinities and NaN."""
    H = 384
    x = torch.zeros(6, H)
    x[1, :128] = 1e18
    x[2, 5] = 1e-30
    x[3] = torch.randn(H, generator=torch.Generator().manual_seed(0))
    x[4, 300] = float("inf")
    x[5, 7] = float("nan")
    w = torch.ones(H)
    for dtype in (BF, F32):
        xd, wd = x.to(dtype).cuda(), w.to(dtype).cuda()
        codes, exps, y, _ = norm.rms_norm_fp8(xd, wd, 1e-6)
        yf = f64(y)
        assert not yf[0].any() and not codes[0].any() and (exps[0] == 127).all()
        assert np.allclose(yf[1, :128], np.sqrt(3), rtol=1e-2) and not yf[1, 128:].any() and exps[1, 1] == 127
        assert np.isfinite(yf[:4]).all()
        rc, re = ox.eight_bits(yf[:4])
        assert np.array_equal(codes[:4].cpu().numpy(), rc) and np.array_equal(exps[:4].cpu().numpy(), re)
        # 1 / inf: the finite columns vanish, the infinite one is none; a NaN takes its row
        assert not yf[4, :300].any() and np.isnan(yf[4, 300]) and np.isnan(yf[5]).all()
        assert (codes[5].cpu() & 127 == 127).all()
        back = norm.fp8_dequantize(codes, exps)
        assert torch.isnan(back[5]).all() and torch.isfinite(back[:4]).all()


def test_large_scale_codes(cuda_device):
    """Scales at both ends of the byte, where y itself is near the ends of float32."""
    H = 256
    g = torch.Generator().manual_seed(3)
    x = torch.randn(4, H, generator=g).cuda()
    for scale in (1e38, 1e-37, 1e-38 / 64):
        w = torch.full((H,), scale, device="cuda") / 4
        codes, exps, y, _ = norm.rms_norm_fp8(x, w, 0.0)
        assert torch.isfinite(y).all()
        rc, re = ox.eight_bits(f64(y))
        assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(exps.cpu().numpy(), re)
        assert np.array_equal(f64(norm.fp8_dequantize(codes, exps, F32)), ox.from_eight_bits(rc, re))


@pytest.mark.parametrize("T,H", [(1, 1), (37, 1), (3, 5), (700, 7), (1, 8), (5, 12), (9, 127), (40, 128), (33, 129), (21, 130), (6, 133), (17, 1111),
                                 (3, 2044), (4, 7168), (2, 16384)])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_every_code_back(cuda_device, T, H, out, shift):
    """All codes and exponents, rows that end inside a unit, bases off the grid."""
    g = torch.Generator().manual_seed(T + H)
    codes = torch.randint(0, 256, (T * H + shift,), generator=g, dtype=torch.uint8).cuda()[shift:].view(T, H)
    exps = torch.randint(0, 256, (T, (H + 127) // 128), generator=g, dtype=torch.uint8).cuda()
    want = torch.from_numpy(ox.from_eight_bits(codes.cpu().numpy(), exps.cpu().numpy()))
    want[(codes.cpu() & 127) == 127] = math.nan
    want[exps.cpu().repeat_interleave(128, 1)[:, :H] == 255] = math.nan
    # four bits are exact but below the range's normal numbers: half a step there
    room = 2.0 ** -134 * (want.abs() < 2.0 ** -126) if out == BF else torch.zeros(T, H)
    want = want.to(out)  # beyond the range: infinity
    for at in (0, shift):
        o = torch.full((T * H + at + 3,), 7.0, dtype=out, device="cuda")
        back = norm.fp8_dequantize(codes, exps, out, o[at:at + T * H].view(T, H)).cpu()
        same = (back == want) | (back.isnan() & want.isnan())
        assert (same | ((back.double() - want.double()).abs() <= room)).all()
        assert (o[:at] == 7).all() and (o[at + T * H:] == 7).all()


@pytest.mark.parametrize("H", [7176, 7177])
def test_codes_beyond_32_bits(cuda_device, H):
    T = 600011
    codes = torch.full((T, H), 0x38, dtype=torch.uint8, device=cuda_device)  # ones
    exps = torch.full((T, (H + 127) // 128), 128, dtype=torch.uint8, device=cuda_device)
    g = torch.Generator().manual_seed(0)
    codes[-9:] = torch.randint(0, 127, (9, H), generator=g, dtype=torch.uint8).cuda()
    exps[-9:] = torch.randint(100, 140, (9, exps.shape[1]), generator=g, dtype=torch.uint8).cuda()
    assert codes.numel() > 2 ** 32
    out = norm.fp8_dequantize(codes, exps)
    assert torch.equal(out[-9:], norm.fp8_dequantize(codes[-9:].clone(), exps[-9:].clone()))
    assert (out[:-9] == 2).all()


@pytest.mark.parametrize("H", [256, 1001])
def test_in_place(cuda_device, H):
    for dtype in (BF, F32):
        x, res, w = make(70, H, dtype)
        y, r = norm.rms_norm(x, w, 1e-6, res)
        x2, r2 = x.clone(), res.clone()
        y2, r2b = norm.rms_norm(x2, w, 1e-6, r2, y=x2, residual_out=r2)
        assert y2 is x2 and r2b is r2 and torch.equal(x2, y) and torch.equal(r2, r)
        dx, dw = norm.rms_norm_backward(x, r, w, 1e-6, res)
        for dst in ("dy", "d_r"):
            a = {"dy": x.clone(), "d_r": res.clone()}
            dx2, dw2 = norm.rms_norm_backward(a["dy"], r, w, 1e-6, a["d_r"], dx=a[dst])
            assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_empty_batch(cuda_device):
    for H in (64, 65):
        x, w = torch.empty(0, H, device="cuda", dtype=BF), torch.ones(H, device="cuda", dtype=BF)
        codes, exps, y, r = norm.rms_norm_fp8(x, w, 1e-6, x)
        assert y.shape == r.shape == codes.shape == (0, H) and exps.shape == (0, 1 if H == 64 else 1)
        dx, dw = norm.rms_norm_backward(x, x, w)
        assert dx.shape == (0, H) and not dw.any()
        assert norm.fp8_dequantize(codes, exps).shape == (0, H)


def test_autograd(cuda_device):
    """Against torch's own differentiation in 64 bits, with and without what reaches r."""
    x, res, w = (t.requires_grad_() for t in make(20, 96, F32))
    up, stream = torch.randn(20, 96, device="cuda"), torch.randn(20, 96, device="cuda")
    for use_r in (True, False):
        for use_y in (True, False):
            if not (use_r or use_y):
                continue
            for added in (True, False):
                for t in (x, res, w):
                    t.grad = None
                y, r = norm.RmsNorm.apply(x, w, 1e-6, res if added else None)
                ((y * up).sum() * use_y + (r * stream).sum() * use_r).backward() if use_r and use_y else \
                    ((y * up).sum() if use_y else (r * stream).sum()).backward()
                xd, rd, wd = (t.detach().double().requires_grad_() for t in (x, res, w))
                q = xd + rd if added else xd + 0
                z = q * wd / (q.square().mean(1, keepdim=True) + 1e-6).sqrt()
                ((z * up).sum() * use_y + (q * stream).sum() * use_r).backward()
                assert torch.allclose(x.grad.double(), xd.grad, atol=1e-5, rtol=1e-5)
                if added:
                    assert torch.allclose(res.grad.double(), rd.grad, atol=1e-5, rtol=1e-5)
                if use_y:
                    assert torch.allclose(w.grad.double(), wd.grad, atol=1e-4, rtol=1e-5)


def test_graph_and_streams(cuda_device):
    """Captured and replayed on new inputs, and on a stream of its own, bit for bit."""
    x, res, w = make(300, 1024, BF)
    dy = make(300, 1024, BF, seed=9)[0]

    def call():
        codes, exps, y, r = norm.rms_norm_fp8(x, w, 1e-6, res)
        return codes, exps, y, r, *norm.rms_norm_backward(dy, r, w, 1e-6, res)

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    codes, exps, y, r = norm.rms_norm_fp8(x, w, 1e-6, res, stream=side)
    dx, dw = norm.rms_norm_backward(dy, r, w, 1e-6, res, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, (codes, exps, y, r, dx, dw)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    x.copy_(make(300, 1024, BF, seed=77)[0])
    graph.replay()
    for a, b in zip(call(), got):
        assert torch.equal(a, b)


def test_offsets_beyond_32_bits(cuda_device):
    T, H = 300007, 7176
    x = torch.empty(T, H, dtype=BF, device="cuda").fill_(0.5)
    tail = make(9, H, BF, seed=4)[0]
    x[-9:] = tail
    w = make(1, H, BF)[2]
    codes, exps, y, _ = norm.rms_norm_fp8(x, w, 1e-6)
    c, e, t, _ = norm.rms_norm_fp8(tail, w, 1e-6)
    assert torch.equal(codes[-9:], c) and torch.equal(exps[-9:], e) and torch.equal(y[-9:], t)
    del codes
    dx, _ = norm.rms_norm_backward(y, x, w, 1e-6, dx=y)
    assert torch.equal(dx[-9:], norm.rms_norm_backward(t, tail, w, 1e-6)[0])
