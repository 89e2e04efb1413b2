"""Microscaled 4-bit quantisation and the experts' product on the GPU.

Codes and scale bytes are decisions and have to be equal to the plain
restatement's.  The product's reference is the 64-bit sum of the codes' values;
its tolerance: one bf16 rounding (2^-8 |ref|) plus, for each of the C / 64 tensor
core steps of float32 accumulation (and two more for the tensor scales), an error
of at most 2^-22 of S = sum |a w|.  Sums whose every partial sum is exact in
float32 have to be exact.
"""
import math

import numpy as np
import pytest
import torch

import lora_moe_expert_info_gb300 as mlr
from lora_moe_expert_info_gb300 import fp4, permute as pm
from oracle import experts as ox

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FMTS = ["mxfp4", "nvfp4"]


def np64(t):
    return t.detach().cpu().double().numpy()


def randn(*shape, seed=0, dtype=F32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def scale_of(x, fmt):
    return None if fmt == "mxfp4" else x.float().abs().max().reshape(1) / 2688


def check_rows(x32, codes, scales, place, fmt, g=1.0):
    """Codes and scales of rows of float32 values against the restatement."""
    rows, cols = x32.shape
    n = 16 if fmt == "nvfp4" else 32
    got = ox.unpack_codes(codes, codes.shape[1] * 2)
    assert not got[:, cols:].any()  # padding codes
    for i in range(rows):
        c, b, _ = ox.quantize_row(x32[i], fmt, g)
        assert np.array_equal(got[i, :cols], c), (i, np.flatnonzero(got[i, :cols] != c))
        blk, r = place(i)
        have = [ox.scale_byte_of(scales, blk, r, j) for j in range(scales.shape[1] * 4)]
        assert have[:b.size] == b.tolist() and not any(have[b.size:])


def matrix_place(i):
    return i // 128, i % 128


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7168), (3, 16), (5, 31), (130, 33), (257, 200), (2, 1001), (40, 72)])
def test_quantize_matrix(cuda_device, fmt, dtype, rows, cols):
    x = randn(rows, cols, seed=rows + cols, dtype=dtype)
    x[0, 0] = -0.0
    g = scale_of(x, fmt)
    codes, scales = fp4.fp4_quantize(x, fmt, g)
    check_rows(x.float().cpu().numpy(), codes.cpu().numpy(), scales.cpu().numpy(), matrix_place, fmt,
               1.0 if g is None else float(g))
    ref = ox.numbers(codes.cpu().numpy(), scales.cpu().numpy(), matrix_place, cols, fmt)
    ref = ref if g is None else ref * float(g)
    for out in (BF, F32):
        y = np64(fp4.fp4_dequantize(codes, scales, cols, fmt, g, dtype=out))
        # code x block scale is exact, then the tensor scale and the output's own rounding
        assert np.all(np.abs(y - ref) <= (2.0 ** -24 + (2.0 ** -8 if out is BF else 2.0 ** -24)) * 1.01 * np.abs(ref))


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_ties_extremes_and_bad_values(cuda_device, fmt):
    f = np.float32
    rows = []
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    for p in (-126, -60, -9, -1, 0, 5, 100):  # ties at every scale, both sides of them
        with np.errstate(over="ignore", under="ignore"):
            t = np.array(ties, dtype=f) * f(2.0) ** f(p)
        rows.append(np.concatenate([t, -t, np.nextafter(t, f(np.inf)), np.nextafter(t, f(0))])[:32])
    rows.append(np.full(32, 3.4028235e38, f))
    rows.append(np.full(32, 1e-45, f))
    rows.append(np.zeros(32, f))
    for bad in (np.inf, -np.inf, np.nan):
        r = np.linspace(-1, 1, 32).astype(f)
        r[5] = bad
        rows.append(r)
    x = np.stack(rows)
    x = np.concatenate([x, x[::-1]], axis=1)
    codes, scales = fp4.fp4_quantize(torch.from_numpy(x).cuda(), fmt)
    check_rows(x, codes.cpu().numpy(), scales.cpu().numpy(), matrix_place, fmt)
    y = fp4.fp4_dequantize(codes, scales, 64, fmt, dtype=F32).cpu().numpy()
    n = 16 if fmt == "nvfp4" else 32
    bad = ~np.isfinite(x).reshape(x.shape[0], -1, n).all(-1)
    assert np.array_equal(np.isnan(y), np.repeat(bad, n, axis=1))


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_stack(cuda_device, fmt):
    E, N, C = 3, 130, 80
    x = randn(E, N, C, seed=1)
    g = x.abs().amax((1, 2)) / 2688 if fmt == "nvfp4" else None
    codes, scales = fp4.fp4_quantize(x, fmt, g)
    assert scales.shape[:2] == (E, 2)
    for e in range(E):
        check_rows(x[e].cpu().numpy(), codes[e].cpu().numpy(), scales[e].cpu().numpy(), matrix_place, fmt,
                   1.0 if g is None else float(g[e]))
    y = fp4.fp4_dequantize(codes, scales, C, fmt, g)
    assert y.shape == (E, N, C)
    one = fp4.fp4_dequantize(codes[1], scales[1], C, fmt, None if g is None else g[1:2])
    assert torch.equal(y[1], one)


def routing(T, K, E, seed=0, masked=0.0, empty=()):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (T, K))
    for e in empty:
        ids[ids == e] = (e + 1) % E
    if masked:
        ids = np.where(rng.random((T, K)) < masked, -1, ids)
    return torch.from_numpy(ids.astype(np.int32)).cuda()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,K,E,C,masked", [(1, 1, 1, 32, 0.0), (1, 8, 16, 208, 0.0), (40, 6, 5, 100, 0.2),
                                            (300, 2, 3, 65, 0.0), (7, 3, 2, 32, 1.0)])
def test_quantize_permuted(cuda_device, fmt, dtype, T, K, E, C, masked):
    x = randn(T, C, seed=T, dtype=dtype)
    ids = routing(T, K, E, seed=C, masked=masked)
    pos, off = pm.moe_sort_pairs(ids, E)
    g = scale_of(x, fmt)
    codes, scales = fp4.fp4_quantize_permuted(x, ids, pos, off, fmt, g, check=True)
    p, o = pos.cpu().numpy(), off.cpu().numpy()
    n = int(o[-1])
    rows = ox.permute(x.float().cpu().numpy(), p)
    assert not codes[n:].any()
    check_rows(rows[:n], codes.cpu().numpy()[:n], scales.cpu().numpy(), ox.sorted_place(o), fmt,
               1.0 if g is None else float(g))
    y = fp4.fp4_dequantize(codes, scales, C, fmt, g, expert_offsets=off)
    direct = fp4.fp4_dequantize(*fp4.fp4_quantize(x, fmt, g), C, fmt, g)
    assert torch.equal(y, pm.moe_permute(direct, ids, E)[0])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 2), (70, 3), (9, 8), (33, 17), (130, 48), (40, 90), (5, 1001), (300, 96)])
def test_any_address(cuda_device, fmt, dtype, rows, cols):
    """Rows at every address their type allows give what rows at a 512-byte
    boundary give, read nothing and write nothing around them."""
    x = randn(rows, cols, seed=cols, dtype=dtype)
    gu = randn(rows, 2 * cols, seed=rows, dtype=dtype)
    off = torch.tensor([0, rows // 3, rows // 3, rows], dtype=torch.int32, device="cuda")
    g = scale_of(x, fmt)
    codes, scales = fp4.fp4_quantize(x, fmt, g)
    back = fp4.fp4_dequantize(codes, scales, cols, fmt, g, dtype=dtype)
    h = fp4.fp4_dequantize(*fp4.fp4_quantize_swiglu(gu, off, fmt, g), cols, fmt, g, expert_offsets=off, dtype=dtype)

    def at(t, k):  # t's values k elements past a boundary, NaN around them
        buf = torch.full((t.numel() + 32,), math.nan, dtype=dtype, device="cuda")
        view = buf[k:k + t.numel()].view(t.shape)
        view.copy_(t)
        return buf, view

    for k in range(16 // x.element_size() + 1):
        c, s = fp4.fp4_quantize(at(x, k)[1], fmt, g)
        assert torch.equal(c, codes)
        r = torch.arange(rows, device="cuda")
        n = scales.shape[1] * 4
        assert torch.equal(scale_bytes(s, r // 128, r % 128, n), scale_bytes(scales, r // 128, r % 128, n))
        buf, out = at(torch.zeros_like(x), k)
        fp4.fp4_dequantize(c, s, cols, fmt, g, dtype=dtype, out=out)
        assert torch.equal(out, back)
        assert buf[:k].isnan().all() and buf[k + x.numel():].isnan().all()
        hk = fp4.fp4_quantize_swiglu(at(gu, k)[1], off, fmt, g)
        assert torch.equal(fp4.fp4_dequantize(*hk, cols, fmt, g, expert_offsets=off, dtype=dtype), h)


def scale_bytes(scales, block, row, count):
    """[rows, count] scale bytes of rows `row` of row blocks `block`."""
    c = torch.arange(count, device=scales.device)
    at = (c // 4) * 512 + (16 * (row % 32) + 4 * (row // 32))[:, None] + c % 4
    return scales.view(scales.shape[0], -1)[block[:, None], at]


@pytest.mark.parametrize("fmt,dtype,T,K,E,C,masked", [
    ("nvfp4", BF, 2100, 8, 40, 7168, 0.0), ("nvfp4", F32, 1300, 12, 300, 7001, 0.1), ("mxfp4", BF, 3300, 9, 7, 7168, 0.3),
    ("mxfp4", F32, 900, 40, 3, 6000, 0.0), ("nvfp4", BF, 4100, 4, 700, 6500, 0.02), ("mxfp4", BF, 80, 200, 5, 16384, 0.0),
    ("nvfp4", BF, 900, 8, 40, 25500, 0.0), ("nvfp4", BF, 900, 8, 40, 25600, 0.0), ("nvfp4", BF, 4000, 8, 2, 3200, 1.0)])
def test_quantize_many_tokens(cuda_device, fmt, dtype, T, K, E, C, masked):
    """Rows of many tokens hold the codes and scales of their tokens quantised
    as a matrix; one expert has no row and one few."""
    x = randn(T, C, seed=T, dtype=dtype)
    ids = routing(T, K, E, seed=C, masked=masked, empty=(1,))
    pos, off = pm.moe_sort_pairs(ids, E)
    g = scale_of(x, fmt)
    codes, scales = fp4.fp4_quantize_permuted(x, ids, pos, off, fmt, g, check=True)
    ref_codes, ref_scales = fp4.fp4_quantize(x, fmt, g)
    n = int(off[-1])
    flat = pos.flatten().long()
    token = torch.arange(T * K, device="cuda") // K
    live = flat >= 0
    src = torch.empty(T * K, dtype=torch.long, device="cuda")
    src[torch.where(live, flat, ~flat)] = token
    assert torch.equal(codes[:n], ref_codes[src[:n]]) and not codes[n:].any()
    r, o = torch.arange(n, device="cuda"), off.long()
    e = torch.searchsorted(o[1:], r, right=True)
    j = r - o[e]
    count = scales.shape[1] * 4
    have = scale_bytes(scales, o[e] // 128 + e + j // 128, j % 128, count)
    assert torch.equal(have, scale_bytes(ref_scales, src[:n] // 128, src[:n] % 128, count))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,K,E,C,masked", [(1, 1, 1, 16, 0.0), (50, 3, 4, 90, 0.2), (200, 2, 3, 64, 0.0), (9, 1, 2, 1001, 0.0)])
def test_quantize_swiglu(cuda_device, fmt, dtype, T, K, E, C, masked):
    """h = u g sigmoid(g) from float32 steps is within 8 x 2^-24 relative of the
    64-bit value (exp, sum, quotient and product of a few ulp each).  The scale
    must be that of a block maximum in that range; each value must then lie
    within half a step of its code, or beyond the largest code."""
    ids = routing(T, K, E, seed=C, masked=masked)
    pos, off = pm.moe_sort_pairs(ids, E)
    P, n = T * K, int(off[-1])
    gu = randn(P, 2 * C, seed=C, dtype=dtype)
    g = torch.full((1,), 24 / 2688, device="cuda") if fmt == "nvfp4" else None
    codes, scales = fp4.fp4_quantize_swiglu(gu, off, fmt, g, check=True)
    assert not codes[n:].any()
    a = np64(gu)
    h = (a[:, :C] / (1 + np.exp(-a[:, :C])) * a[:, C:])[:n]
    place = ox.sorted_place(off.cpu().numpy())
    sc = scales.cpu().numpy()
    num = ox.numbers(codes.cpu().numpy()[:n], sc, place, C, fmt) * (1.0 if g is None else float(g))
    val = ox.unpack_scales(sc, place, n, C, fmt) * (1.0 if g is None else float(g))
    w = 16 if fmt == "nvfp4" else 32
    eps = 8 * 2.0 ** -24
    for i in range(n):
        b, r = place(i)
        for c in range(0, C, w):
            most = np.abs(h[i, c:c + w]).max()
            byte = ox.scale_byte_of(sc, b, r, c // w)
            g1 = 1.0 if g is None else float(g)
            assert byte in {ox.block_scale(float(np.float32(most * k)), fmt, g1)[0] for k in (1 - eps, 1, 1 + eps)}
    s = np.repeat(val, w, axis=1)[:, :C]
    q = np.abs(num) / np.where(s > 0, s, 1)
    up = np.where(q < 2, 0.25, np.where(q < 4, 0.5, 1.0))  # half a step above the code's value
    dn = np.where(q <= 2, 0.25, np.where(q <= 4, 0.5, 1.0))
    v = np.sign(num) * h
    v = np.where(num == 0, np.abs(h), v) / np.where(s > 0, s, 1)
    slack = 1e-5 * np.maximum(v, 1)
    ok = (v >= q - dn - slack) & ((v <= q + up + slack) | (q == 6)) | (s == 0)
    assert ok.all()


def product_case(T, K, E, N, C, fmt, seed=0, masked=0.0, empty=()):
    ids = routing(T, K, E, seed=seed, masked=masked, empty=empty)
    pos, off = pm.moe_sort_pairs(ids, E)
    x = randn(T, C, seed=seed)
    w = randn(E, N, C, seed=seed + 1) / math.sqrt(C)
    ga = scale_of(x, fmt)
    gw = w.abs().amax((1, 2)) / 2688 if fmt == "nvfp4" else None
    a, sa = fp4.fp4_quantize_permuted(x, ids, pos, off, fmt, ga)
    qw, sw = fp4.fp4_quantize(w, fmt, gw)
    return off, a, sa, qw, sw, ga, gw


def product_reference(off, a, sa, qw, sw, ga, gw, C, fmt):
    """(y, S) in 64 bits from the dequantised operands (their own tests hold them
    to the restatement; float32 dequantisation without a tensor scale is exact)."""
    P, N = a.shape[0], qw.shape[1]
    y, S = torch.zeros(P, N, dtype=torch.float64), torch.zeros(P, N, dtype=torch.float64)
    av = fp4.fp4_dequantize(a, sa, C, fmt, expert_offsets=off, dtype=F32).double()
    wv = fp4.fp4_dequantize(qw, sw, C, fmt, dtype=F32).double()
    o = off.tolist()
    for e in range(qw.shape[0]):
        if o[e + 1] > o[e]:
            g = 1.0 if ga is None else float(ga) * float(gw[e])
            r = slice(o[e], o[e + 1])
            y[r] = (av[r] @ wv[e].T * g).cpu()
            S[r] = (av[r].abs() @ wv[e].abs().T * g).cpu()
    return y.numpy(), S.numpy()


def check_product(off, a, sa, qw, sw, ga, gw, C, fmt):
    y = fp4.fp4_expert_product(a, sa, off, qw, sw, C, fmt, ga, gw)
    ref, S = product_reference(off, a, sa, qw, sw, ga, gw, C, fmt)
    err = np.abs(np64(y) - ref) - (2.0 ** -8 * np.abs(ref) + (C / 64 + 2) * 2.0 ** -22 * S)
    assert np.all(err <= 0), f"outside by {err.max()} at {np.unravel_index(err.argmax(), err.shape)}"
    return y


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,K,E,N,C,masked", [
    (1, 1, 1, 1, 1, 0.0), (1, 1, 1, 128, 64, 0.0), (1, 8, 16, 200, 7168, 0.0), (16, 1, 1, 64, 96, 0.0), (17, 2, 3, 130, 100, 0.0),
    (60, 3, 4, 129, 257, 0.2), (128, 1, 1, 256, 256, 0.0), (129, 1, 1, 256, 288, 0.0), (255, 1, 1, 127, 31, 0.0),
    (256, 1, 1, 128, 512, 0.0), (257, 1, 1, 384, 64, 0.0), (700, 1, 2, 96, 320, 0.0), (300, 8, 5, 264, 768, 0.1),
    (513, 2, 300, 72, 128, 0.0), (5, 2, 3, 128, 128, 1.0)])
def test_product(cuda_device, fmt, T, K, E, N, C, masked):
    check_product(*product_case(T, K, E, N, C, fmt, seed=T + C, masked=masked), C, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_product_with_empty_experts(cuda_device, fmt):
    check_product(*product_case(40, 2, 9, 160, 192, fmt, seed=3, empty=(0, 4, 5, 8)), 192, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows", [65, 128, 129, 192, 200, 257, 700])
def test_product_with_one_long_expert(cuda_device, fmt, rows):
    """Few rows per expert on average, many for one: its row tiles begin inside
    the 128-row blocks of its scales."""
    E = 40
    ids = torch.cat([torch.arange(E), torch.full((rows,), 7)]).to(torch.int32).cuda().view(-1, 1)
    pos, off = pm.moe_sort_pairs(ids, E)
    x = randn(ids.shape[0], 320, seed=rows)
    w = randn(E, 136, 320, seed=rows + 1)
    check_product(off, *fp4.fp4_quantize_permuted(x, ids, pos, off, fmt), *fp4.fp4_quantize(w, fmt), None, None, 320, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,E,N,C", [(1, 1, 256, 4096), (33, 2, 300, 1000), (400, 1, 130, 544), (1000, 3, 257, 2048)])
def test_product_exact_sums(cuda_device, fmt, T, E, N, C):
    """Scales 2^-1..2^1 and codes give products that are multiples of 2^-4 and
    sums below 2^20: every partial sum is exact in float32, so y is the exact
    sum rounded once."""
    rng = np.random.default_rng(T)
    ids = routing(T, 1, E, seed=T)
    _, off = pm.moe_sort_pairs(ids, E)

    def random(rows, blocks, seed):
        g = torch.Generator().manual_seed(seed)
        codes = torch.randint(0, 256, (*rows, (C + 31) // 32 * 16), generator=g, dtype=torch.uint8)
        if C % 32:  # zero codes past the last column
            q = torch.from_numpy(ox.unpack_codes(codes.reshape(-1, codes.shape[-1]).numpy(), 2 * codes.shape[-1]).copy())
            q[:, C:] = 0
            codes = (q[:, 0::2] | q[:, 1::2] << 4).reshape(codes.shape)
        atoms = -(-C // (64 if fmt == "nvfp4" else 128))
        e = torch.randint(-1, 2, (*blocks, atoms, 32, 4, 4), generator=g)
        sc = (e + 127) if fmt == "mxfp4" else (e + 7) * 8
        return codes.cuda(), sc.to(torch.uint8).cuda()

    a, sa = random((T,), (T // 128 + E,), 1)
    w, sw = random((E, N), (E, (N + 127) // 128), 2)
    y = fp4.fp4_expert_product(a, sa, off, w, sw, C, fmt)
    ref, S = product_reference(off, a, sa, w, sw, None, None, C, fmt)
    assert S.max() < 2 ** 20
    assert torch.equal(y.cpu().float(), torch.from_numpy(ref).float().bfloat16().float())


@pytest.mark.parametrize("fmt", FMTS)
def test_product_bad_blocks_stay_in_their_rows(cuda_device, fmt):
    """A NaN scale in one row or one weight row makes that row or column of y
    NaN and nothing else; rows of other experts and scales of rows that do not
    exist reach no result."""
    off, a, sa, qw, sw, ga, gw = product_case(150, 1, 2, 140, 96, fmt, seed=5)
    y0 = fp4.fp4_expert_product(a, sa, off, qw, sw, 96, fmt, ga, gw)
    nan = 0xFF if fmt == "mxfp4" else 0x7F
    o = off.tolist()
    # scales of rows past the experts' last ones
    sa2 = sa.clone()
    for e in range(2):
        n = o[e + 1] - o[e]
        for j in range(n, (n + 127) // 128 * 128):
            sa2[o[e] // 128 + e + j // 128, :, j % 32, j % 128 // 32] = nan
    sw2 = sw.clone()
    for r in range(140, 256):
        sw2[:, r // 128, :, r % 32, r % 128 // 32] = nan
    assert torch.equal(y0, fp4.fp4_expert_product(a, sa2, off, qw, sw2, 96, fmt, ga, gw))
    sa2[o[1] // 128 + 1, 0, 3, 0, 1] = nan  # row 3 of expert 1
    sw2[0, 1, 0, 2, 0, 0] = nan             # output 130 of expert 0
    y = fp4.fp4_expert_product(a, sa2, off, qw, sw2, 96, fmt, ga, gw)
    want = torch.zeros_like(y, dtype=torch.bool)
    want[o[1] + 3] = True
    want[:o[1], 130] = True
    assert torch.equal(y.isnan(), want) and torch.equal(y[~want], y0[~want])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_swiglu_of_bad_and_extreme_values(cuda_device, fmt, bad):
    """A block with an infinity or a NaN is NaN and leaves its neighbours alone;
    gates far below zero give zeros, far above the other factor."""
    P, C = 6, 64
    gu = torch.ones(P, 2 * C)
    gu[0, 5] = bad
    gu[1, C + 40] = bad
    gu[2, :C], gu[2, C:] = -200.0, 3.0   # SiLU -> 0
    gu[3, :C], gu[3, C:] = -88.0, 3.0
    gu[4, :C], gu[4, C:] = 100.0, 0.0    # u = 0
    gu[5, :C], gu[5, C:] = 96.0, 0.5     # 48 in float32
    off = torch.tensor([0, P], dtype=torch.int32, device="cuda")
    codes, scales = fp4.fp4_quantize_swiglu(gu.cuda(), off, fmt, check=True)
    y = fp4.fp4_dequantize(codes, scales, C, fmt, expert_offsets=off, dtype=F32).cpu()
    n = 16 if fmt == "nvfp4" else 32
    want = torch.zeros(P, C, dtype=torch.bool)
    # -inf as a gate: -inf / inf is NaN as well
    want[0, 0:n] = True
    want[1, 40 // n * n:40 // n * n + n] = True
    assert torch.equal(y.isnan(), want)
    assert (y[2:5].abs() < 1e-30).all() and (y[5] == 48).all()


def test_product_rejects_bad_offsets(cuda_device):
    off, a, sa, qw, sw, _, _ = product_case(20, 1, 3, 128, 64, "mxfp4")
    for bad in ([0, 5, 3, 20], [-1, 5, 9, 20], [0, 5, 9, 21]):
        with pytest.raises(mlr.MoeLoraError) as ei:
            fp4.fp4_expert_product(a, sa, torch.tensor(bad, dtype=torch.int32, device="cuda"), qw, sw, 64, "mxfp4")
        assert ei.value.code == mlr.MLR_ERR_INDEX


def test_permuted_rejects_places_of_another_order(cuda_device):
    x = randn(20, 64)
    ids = routing(20, 2, 4, seed=1)
    pos, off = pm.moe_sort_pairs(ids, 4)
    for p in (pos + 40, pos.flip(0).contiguous()):
        with pytest.raises(mlr.MoeLoraError):
            fp4.fp4_quantize_permuted(x, ids, p, off, "mxfp4", check=True)
    with pytest.raises(mlr.MoeLoraError):
        fp4.fp4_quantize_permuted(x, ids + 4, pos, off, "mxfp4", check=True)


def test_unaligned_input_rows(cuda_device):
    base = randn(20 * 64 + 1, dtype=BF)
    x = base[1:].view(20, 64)
    for fmt in FMTS:
        a, b = fp4.fp4_quantize(x, fmt), fp4.fp4_quantize(x.clone(), fmt)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1].flatten(1)[:, :20 * 16], b[1].flatten(1)[:, :20 * 16]) or \
            torch.equal(fp4.fp4_dequantize(*a, 64, fmt), fp4.fp4_dequantize(*b, 64, fmt))


def test_no_rows(cuda_device):
    x = torch.empty(0, 64, device="cuda", dtype=BF)
    codes, scales = fp4.fp4_quantize(x, "nvfp4")
    assert codes.shape == (0, 32) and fp4.fp4_dequantize(codes, scales, 64, "nvfp4").shape == (0, 64)
    ids = torch.empty(0, 2, device="cuda", dtype=torch.int32)
    pos, off = pm.moe_sort_pairs(ids, 3)
    a, sa = fp4.fp4_quantize_permuted(x, ids, pos, off)
    w, sw = fp4.fp4_quantize(randn(3, 16, 64))
    assert fp4.fp4_expert_product(a, sa, off, w, sw, 64).shape == (0, 16)


def test_side_stream_and_repeats(cuda_device):
    args = product_case(200, 4, 6, 192, 320, "nvfp4", seed=2)
    off, a, sa, qw, sw, ga, gw = args
    y = fp4.fp4_expert_product(a, sa, off, qw, sw, 320, "nvfp4", ga, gw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.full_like(y, 3)
    for _ in range(3):
        fp4.fp4_expert_product(a, sa, off, qw, sw, 320, "nvfp4", ga, gw, y=out, stream=s, check=False)
    s.synchronize()
    assert torch.equal(out, y)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,K,E,H,I,masked", [(1, 2, 8, 256, 512, 0.0), (64, 2, 8, 256, 512, 0.1), (300, 4, 6, 1000, 72, 0.0)])
def test_layer(cuda_device, fmt, T, K, E, H, I, masked):
    """fp4_moe_forward against a 64-bit layer on the dequantised weights.  Every
    activation rounded to 4 bits is off by at most a sixth of its block's
    maximum over the block; at random signs the relative error of each of the
    two products is about 0.1, and the layer's below 0.25 in the 2-norm."""
    x = randn(T, H, seed=1, dtype=BF)
    ids = routing(T, K, E, seed=2, masked=masked)
    tw = torch.rand(T, K, generator=torch.Generator().manual_seed(3)).cuda()
    wg, wd = randn(E, 2 * I, H, seed=4) / math.sqrt(H), randn(E, H, I, seed=5) / math.sqrt(I)
    nv = fmt == "nvfp4"
    gg, gd = (wg.abs().amax((1, 2)) / 2688, wd.abs().amax((1, 2)) / 2688) if nv else (None, None)
    qg, qd = fp4.fp4_quantize(wg, fmt, gg), fp4.fp4_quantize(wd, fmt, gd)
    gx = scale_of(x, fmt)
    gh = torch.full((1,), 24 / 2688, device="cuda") if nv else None
    y = fp4.fp4_moe_forward(x, ids, tw, *qg, *qd, fmt, gg, gd, gx, gh)
    g64 = np64(fp4.fp4_dequantize(*qg, H, fmt, gg, dtype=F32))
    d64 = np64(fp4.fp4_dequantize(*qd, I, fmt, gd, dtype=F32))
    ref = np.zeros((T, H))
    for t in range(T):
        for k in range(K):
            e = int(ids[t, k])
            if e >= 0:
                a = g64[e] @ np64(x[t])
                h = a[:I] / (1 + np.exp(-a[:I])) * a[I:]
                ref[t] += float(tw[t, k]) * (d64[e] @ h)
    assert np.linalg.norm(np64(y) - ref) <= 0.25 * np.linalg.norm(ref)
    # and step by step, exactly
    pos, off = pm.moe_sort_pairs(ids, E)
    a, sa = fp4.fp4_quantize_permuted(x, ids, pos, off, fmt, gx)
    gu = fp4.fp4_expert_product(a, sa, off, *qg, H, fmt, gx, gg)
    h, sh = fp4.fp4_quantize_swiglu(gu, off, fmt, gh)
    d = fp4.fp4_expert_product(h, sh, off, *qd, I, fmt, gh, gd)
    assert torch.equal(y, pm.moe_unpermute(d, pos, tw))
