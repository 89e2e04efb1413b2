"""The sorted rows, their gradients and the 4-bit experts used together: the
example, the layer in a CUDA graph and on a side stream, and the product's
bounded waits."""
import math
import os
import sys

import numpy as np
import pytest
import torch

import lora_moe_expert_info_gb300 as mlr
from lora_moe_expert_info_gb300 import fp4, permute as pm
from test_gpu_fp4 import randn, routing, scale_of

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer  # noqa: E402

pytestmark = pytest.mark.gpu
DEFAULT_NS = 2_000_000_000


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_example_trains_and_serves(cuda_device, fmt):
    """The teacher is 1.5 times the layer, which adapters and weights can follow:
    the loss has to fall.  Weights and activations of 4 bits are each off by
    about a tenth, in two products one after the other: 0.3 bounds the layer."""
    losses, prompt, token = expert_layer.run(steps=12, fmt=fmt)
    assert losses[-1] < 0.8 * losses[0]
    assert prompt < 0.3 and token < 0.4


def test_example_gradients_match_dense_autograd(cuda_device):
    """The example's gradients against the same layer written densely in float64:
    bf16 rows and products are each rounded to 2^-8, a few of them in a row."""
    layer = expert_layer.ExpertLayer(4, 2, 64, 96, 4, seed=3)
    with torch.no_grad():
        layer.b_gate_up.normal_(std=0.05, generator=torch.Generator("cuda").manual_seed(1))
        layer.b_down.normal_(std=0.05, generator=torch.Generator("cuda").manual_seed(2))
    x = randn(40, 64, seed=4, dtype=torch.bfloat16).requires_grad_()
    dy = randn(40, 64, seed=5, dtype=torch.bfloat16)
    layer(x).backward(dy)
    got = [x.grad] + [p.grad for p in layer.parameters()]

    params = [p.detach().double().requires_grad_() for p in layer.parameters()]
    router, a1, b1, a2, b2 = params
    xd = x.detach().double().requires_grad_()
    ids, _ = expert_layer.route(x.detach(), layer.router.detach(), 2)
    p = (xd @ router).softmax(-1).gather(1, ids.long())
    w = p / p.sum(-1, keepdim=True)
    gu, dn = layer.w_gate_up.double() + b1 @ a1, layer.w_down.double() + b2 @ a2
    h = torch.einsum("th,enh->ten", xd, gu)
    g, u = h.chunk(2, -1)
    y = torch.einsum("ten,ehn->teh", torch.nn.functional.silu(g) * u, dn)
    mask = torch.zeros(40, 4, dtype=torch.float64, device="cuda").scatter(1, ids.long(), 1.0)
    wide = torch.zeros_like(mask).scatter(1, ids.long(), w) * mask
    (y * wide[..., None]).sum(1).backward(dy.double())
    for name, a, b in zip(["x", "router", "a1", "b1", "a2", "b2"], got, [xd.grad] + [q.grad for q in params]):
        err = float((a.double() - b).norm() / b.norm())
        assert err < 8 * 2.0 ** -8, (name, err)


def layer_case(T, K, E, H, I, fmt="nvfp4"):
    nv = fmt == "nvfp4"
    wg, wd = randn(E, 2 * I, H, seed=4) / math.sqrt(H), randn(E, H, I, seed=5) / math.sqrt(I)
    gg, gd = (wg.abs().amax((1, 2)) / 2688, wd.abs().amax((1, 2)) / 2688) if nv else (None, None)
    x = randn(T, H, seed=1, dtype=torch.bfloat16)
    tw = torch.rand(T, K, generator=torch.Generator().manual_seed(3)).cuda()
    return (x, routing(T, K, E, seed=2), tw, *fp4.fp4_quantize(wg, fmt, gg), *fp4.fp4_quantize(wd, fmt, gd), fmt, gg, gd,
            scale_of(x, fmt), torch.full((1,), 24 / 2688, device="cuda") if nv else None)


@pytest.mark.parametrize("T", [1, 200])
def test_layer_graph_replay_and_side_stream(cuda_device, T):
    args = layer_case(T, 4, 8, 256, 320)
    y0 = fp4.fp4_moe_forward(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert torch.equal(y0, fp4.fp4_moe_forward(*args, stream=s))
    y = torch.empty_like(y0)
    with torch.cuda.stream(s):
        fp4.fp4_moe_forward(*args, y=y, check=False)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fp4.fp4_moe_forward(*args, y=y, check=False)
    args[0].copy_(args[0].flip(0).neg())
    args[1].copy_(args[1].flip(1))
    y.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, fp4.fp4_moe_forward(*args))


@pytest.mark.parametrize("rows,experts", [(1200, 40), (5000, 40)])
def test_product_waits_give_up_then_recover(cuda_device, rows, experts):
    """With a limit of 1 ns the first wait that the device's timer sees take any
    time gives up: the call returns with the status bit, and the next one, with
    the limit put back, is right.  Both row-tile shapes, long enough for waits
    to outlast the timer's steps."""
    C, N = 7168, 2048
    g = torch.Generator("cuda").manual_seed(0)

    def random(rows, blocks):
        codes = torch.randint(0, 256, (*rows, C // 2), generator=g, device="cuda", dtype=torch.uint8)
        return codes, torch.full((*blocks, C // 64, 32, 4, 4), 56, device="cuda", dtype=torch.uint8)

    off = (torch.arange(experts + 1, device="cuda", dtype=torch.int32) * (rows // experts)).contiguous()
    args = (*random((rows,), (rows // 128 + experts,)), off, *random((experts, N), (experts, N // 128)), C, "nvfp4")
    y0 = fp4.fp4_expert_product(*args)
    assert mlr.wait_limit_ns() == DEFAULT_NS
    mlr.set_wait_limit_ns(0)
    try:
        with pytest.raises(mlr.MoeLoraError) as ei:
            fp4.fp4_expert_product(*args)
        assert ei.value.code == mlr.MLR_ERR_TIMEOUT
    finally:
        mlr.set_wait_limit_ns(DEFAULT_NS)
    for _ in range(2):
        assert torch.equal(y0, fp4.fp4_expert_product(*args))


def test_layer_rejects_inconsistent_arguments(cuda_device):
    args = list(layer_case(8, 2, 4, 128, 64))
    with pytest.raises(ValueError):
        fp4.fp4_moe_forward(*args[:5], args[5][:3].contiguous(), *args[6:])
    with pytest.raises(TypeError):
        fp4.fp4_moe_forward(args[0].float(), *args[1:])
    with pytest.raises(ValueError):
        fp4.fp4_moe_forward(*args[:7], "int4", *args[8:])
    bad = args[1].clone()
    bad[0, 0] = 9
    with pytest.raises(mlr.MoeLoraError):
        fp4.fp4_moe_forward(args[0], bad, *args[2:])
    assert np.isfinite(fp4.fp4_moe_forward(args[0], bad.clamp(max=-1), *args[2:]).float().cpu().numpy()).all()
