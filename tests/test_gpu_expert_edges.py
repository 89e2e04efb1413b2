"""Corners of the expert operators' arguments: buffers at every address their type
allows, buffers of the caller that the kernels cannot write, waits that give up, gates far
below zero."""
import math
import threading
import time

import numpy as np
import pytest
import torch

import lora_moe_expert_info_gb300 as mlr
from lora_moe_expert_info_gb300 import fp4, permute as pm
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


def test_buffers_of_the_caller_on_the_host_are_refused(cuda_device):
    """A workspace or a status word that the kernels would write, on the host, with
    holes or too small; a workspace may have any type."""
    ids = torch.zeros(9000, 2, dtype=torch.int32, device="cuda")
    n = pm._lib().moe_permute_workspace_bytes(9000, 2, 4)
    want = pm.moe_sort_pairs(ids, 4)
    got = pm.moe_sort_pairs(ids, 4, workspace=torch.empty((n + 3) // 4, device="cuda"))
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    for ws, error in ((torch.empty(n, dtype=torch.uint8), ValueError), (n, TypeError),
                      (torch.empty(n - 1, dtype=torch.uint8, device="cuda"), mlr.MoeLoraError),
                      (torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2], ValueError)):
        with pytest.raises(error):
            pm.moe_sort_pairs(ids, 4, workspace=ws)
    off, a, sa, qw, sw, ga, gw = product_case(20, 1, 3, 128, 64, "mxfp4")
    with pytest.raises(ValueError):
        fp4.fp4_expert_product(a, sa, off, qw, sw, 64, "mxfp4", status=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        fp4.fp4_expert_product(a, sa, off, qw, sw, 64, "mxfp4", status=torch.zeros(1, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    fp4.fp4_expert_product(a, sa, off, qw, sw, 64, "mxfp4", status=status, check=False)
    assert int(status) == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,experts", [(1200, 40), (5000, 40)])
def test_product_that_gives_up_leaves_nothing_behind(cuda_device, fmt, rows, experts):
    """Waits that give up anywhere between the first step and the last: what was
    issued by then is waited for, which takes microseconds (the waits of the
    teardown, for copies and MMAs, run out after two seconds each: a call that
    needs one of them is a failure), and a product launched right behind, into
    the same shared memory and TMEM, is right."""
    C, N = 7168, 2048
    g = torch.Generator("cuda").manual_seed(0)

    def random(rows, blocks):
        codes = torch.randint(0, 256, (*rows, C // 2), generator=g, device="cuda", dtype=torch.uint8)
        byte = 56 if fmt == "nvfp4" else 127
        return codes, torch.full((*blocks, C // (64 if fmt == "nvfp4" else 128), 32, 4, 4), byte, device="cuda",
                                 dtype=torch.uint8)

    off = (torch.arange(experts + 1, device="cuda", dtype=torch.int32) * (rows // experts)).contiguous()
    args = (*random((rows,), (rows // 128 + experts,)), off, *random((experts, N), (experts, N // 128)), C, fmt)
    want = fp4.fp4_expert_product(*args)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gave_up = 0
    default = mlr.wait_limit_ns()
    try:
        for limit in (0, 300, 600, 1000, 1500, 2000, 3000, 5000, 8000, 20000) * 3:
            status.zero_()
            torch.cuda.synchronize()
            t0 = time.monotonic()
            mlr.set_wait_limit_ns(limit)
            y = fp4.fp4_expert_product(*args, status=status, check=False)
            mlr.set_wait_limit_ns(default)
            behind = fp4.fp4_expert_product(*args, check=False)
            bits = int(status)
            assert time.monotonic() - t0 < 1
            assert bits in (0, 0x10) and torch.equal(behind, want)
            assert bits or torch.equal(y, want)
            gave_up += bits != 0
    finally:
        mlr.set_wait_limit_ns(default)
    assert gave_up


@pytest.mark.parametrize("T,K,E", [(1025, 8, 60), (2048, 8, 60), (16384, 1, 16384)])
def test_order_alone_needs_no_workspace(cuda_device, T, K, E):
    """Between the largest single launch with rows and without: null is taken for
    the order alone, nothing is allocated for it, and rows still need theirs."""
    ids = torch.randint(-1, E, (T, K), generator=torch.Generator().manual_seed(T), dtype=torch.int32).cuda()
    x = torch.zeros(T, 8, device="cuda")
    rows, want, first = pm.moe_permute(x, ids, E)
    pos, off = torch.empty_like(want), torch.empty_like(first)
    f = pm._lib().moe_permute
    stream = torch.cuda.current_stream().cuda_stream
    assert f(None, ids.data_ptr(), T, K, 0, E, 0, None, pos.data_ptr(), off.data_ptr(), None, 0, None, stream) == mlr.MLR_OK
    assert torch.equal(pos, want) and torch.equal(off, first)
    assert f(x.data_ptr(), ids.data_ptr(), T, K, 8, E, 1, rows.data_ptr(), pos.data_ptr(), off.data_ptr(), None, 0, None,
             stream) == mlr.MLR_ERR_CAPACITY
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    pm.moe_sort_pairs(ids, E, pair_pos=pos, expert_offsets=off, check=False)
    assert torch.cuda.max_memory_allocated() == before


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gate,up", [(-85.9, 3e38), (-86.1, 3e38), (-86.5, 1e38), (-88.0, 3e38), (-89.0, -3e38), (-95.0, 3e38),
                                     (-100.0, 3e38), (-103.5, 3e38), (-120.0, 3e38), (-168.0, 3e38), (-1e4, 3e38),
                                     (-1e30, 3e38), (-3e38, 1.0), (-3e38, -3e38), (-88.0, 1.0), (-100.0, 1.0)])
def test_swiglu_of_gates_far_below_zero(cuda_device, fmt, gate, up):
    """u g / (1 + exp(-g)) where 1 / (1 + exp(-g)) is no normal float, or none at
    all: blocks of one value, whose 4-bit number is within a fifth of it (the value
    5 between the codes 4 and 6; float32 steps add less than a hundredth of that)
    or, below the smallest scale, half of its smallest code (MXFP4) or that scale
    (NVFP4).  Gates of zero among them give zeros."""
    g32 = float(np.float32(gate))
    h = g32 * math.exp(g32) / (1 + math.exp(g32)) * float(np.float32(up))
    block = 16 if fmt == "nvfp4" else 32
    most = max(abs(h), 1e-30)
    scale = torch.tensor([most / 2688], device="cuda") if fmt == "nvfp4" else None
    gu = torch.full((2, 4 * block), 0.0)
    gu[0, :2 * block], gu[0, 2 * block:] = gate, up
    gu[1, 0:2 * block:2], gu[1, 1:2 * block:2] = gate, 0.0   # beside gates of 0
    gu[1, 2 * block::2], gu[1, 2 * block + 1::2] = up, 1.0
    off = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    codes, scales = fp4.fp4_quantize_swiglu(gu.cuda(), off, fmt, scale, check=True)
    y = fp4.fp4_dequantize(codes, scales, 2 * block, fmt, scale, expert_offsets=off, dtype=torch.float32)
    y = y.cpu().double().numpy()
    floor = 2.0 ** -127 / 4 if fmt == "mxfp4" else 2.0 ** -9 * float(scale)
    assert (np.abs(y[0] - h) <= 0.202 * abs(h) + 1.01 * floor).all(), (y[0, 0], h)
    assert (np.abs(y[1, 0::2] - h) <= 0.202 * abs(h) + 1.01 * floor).all()
    assert not y[1, 1::2].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rows,cols", [(70, 128), (33, 90), (5, 7168), (9, 1001)])
def test_swiglu_blocks_with_far_gates_leave_the_others_alone(cuda_device, fmt, dtype, rows, cols):
    """Some blocks hold a far gate, an infinity or a NaN: all others have the codes
    and scales that they have without those, whatever the row's vectors."""
    g = torch.Generator().manual_seed(cols)
    gu = torch.randn(rows, 2 * cols, generator=g)
    bad = gu.clone()
    n = 16 if fmt == "nvfp4" else 32
    touched = torch.zeros(rows, -(-cols // n) * n, dtype=torch.bool)
    for value in (-90.0, -3e38, math.inf, math.nan):
        for _ in range(3):
            r, c = (int(torch.randint(m, (1,), generator=g)) for m in (rows, cols))
            bad[r, c] = value
            touched[r, c // n * n:c // n * n + n] = True
    far = touched & (torch.nn.functional.pad(bad[:, :cols], (0, touched.shape[1] - cols)).isfinite().view(rows, -1, n)
                     .all(-1, keepdim=True).expand(-1, -1, n).reshape(touched.shape))
    off = torch.tensor([0, rows // 3, rows // 3, rows], dtype=torch.int32, device="cuda")
    y = [fp4.fp4_dequantize(*fp4.fp4_quantize_swiglu(t.to(dtype).cuda(), off, fmt, check=True), cols, fmt, expert_offsets=off,
                            dtype=torch.float32).cpu() for t in (gu, bad)]
    touched, far = touched[:, :cols], far[:, :cols]
    assert torch.equal(y[0][~touched], y[1][~touched])
    assert torch.equal(y[1].isnan(), touched & ~far)
    # in blocks with far gates those are zero and the others within half a code's step of the block's scale
    h = torch.nn.functional.silu(bad[:, :cols].to(dtype).double()) * bad[:, cols:].to(dtype).double()
    most = torch.nn.functional.pad(h.abs(), (0, -cols % n)).view(rows, -1, n).amax(-1, keepdim=True)
    step = (most / 3).expand(-1, -1, n).reshape(rows, -1)[:, :cols]
    assert bool(((y[1] - h).abs()[far] <= step[far] + 2.0 ** -9).all())


@pytest.mark.parametrize("T,experts", [(40, (16384, 5200)), (9000, (16384, 12500))])
def test_sorts_of_different_experts_in_two_threads(cuda_device, T, experts):
    """Each thread's launches need another amount of shared memory of the same
    kernels (in one launch, and counted first); none takes the other's away."""
    lib = pm._lib()
    codes, done = [], []

    def sort(E):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            ids = (torch.arange(T, dtype=torch.int32, device="cuda") * 7 % E).view(T, 1)
            x = torch.arange(T, dtype=torch.float32, device="cuda").view(T, 1).expand(T, 8).contiguous()
            rows, pos = torch.empty_like(x), torch.empty_like(ids)
            off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
            ws = torch.empty(lib.moe_permute_workspace_bytes(T, 1, E), dtype=torch.uint8, device="cuda")
            for _ in range(3000):
                codes.append(lib.moe_permute(x.data_ptr(), ids.data_ptr(), T, 1, 8, E, 1, rows.data_ptr(), pos.data_ptr(),
                                             off.data_ptr(), ws.data_ptr(), ws.nbytes, None, s.cuda_stream))
            s.synchronize()
            done.append(torch.equal(rows[pos.view(-1).long()], x))

    threads = [threading.Thread(target=sort, args=(E,)) for E in experts]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert codes == [mlr.MLR_OK] * 6000 and done == [True, True]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("P,E,N,first,last", [(40, 3, 128, 7, 33), (700, 2, 129, 130, 700), (9, 4, 64, 9, 9), (2000, 2, 72, 1000, 1999)])
def test_rows_before_the_first_expert(cuda_device, fmt, P, E, N, first, last):
    """Offsets need not begin at 0: rows before the first expert's are no expert's,
    as are those past the last one's.  Their codes and results are zeros, and
    the others are those of the same rows alone."""
    C = 96
    off = torch.linspace(first, last, E + 1).int().cuda()
    gu = torch.randn(P, 2 * C, generator=torch.Generator().manual_seed(P)).cuda()
    codes = torch.full((P, 48), 255, dtype=torch.uint8, device="cuda")
    codes, scales = fp4.fp4_quantize_swiglu(gu, off, fmt, codes=codes, check=True)
    assert not codes[:first].any() and not codes[last:].any()
    h = fp4.fp4_dequantize(codes, scales, C, fmt, expert_offsets=off, dtype=torch.float32)
    assert not h[:first].any() and not h[last:].any()
    qw, sw = fp4.fp4_quantize(torch.randn(E, N, C, generator=torch.Generator().manual_seed(N)).cuda(), fmt)
    y = torch.full((P, N), 7.0, dtype=BF, device="cuda")
    fp4.fp4_expert_product(codes, scales, off, qw, sw, C, fmt, y=y)
    assert not y[:first].any() and not y[last:].any()
    if first < last:
        part = fp4.fp4_quantize_swiglu(gu[first:last].contiguous(), off - first, fmt, check=True)
        assert torch.equal(part[0], codes[first:last])
        assert torch.equal(fp4.fp4_expert_product(*part, off - first, qw, sw, C, fmt), y[first:last])
