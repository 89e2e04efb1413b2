"""The operators before the experts used together with the layers that follow them."""
import threading

import numpy as np
import pytest
import torch

import lora_moe_expert_info_gb300 as mlr
from lora_moe_expert_info_gb300 import fp4, norm, permute as pm, router as rt
from test_gpu_forward import custom_case, workload_case
from test_gpu_quant import LORA
from test_gpu_w8a8 import quant_of

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def layer(c, q, x, ids, w, **kw):
    lo = [getattr(c.w, k) for k in LORA]
    mapping = torch.from_numpy(np.asarray(c.mapping, dtype=np.int32)).to(x.device)
    return mlr.fused_moe_lora_forward_fp8_w8a8(x, ids, w, mapping, c.b.lora_ranks, c.scal, q.w_gate_up_q, q.w_gate_up_exp,
                                               q.w_down_q, q.w_down_exp, *lo, **kw)


# rows copied pair by pair and token by token, hidden sizes that end inside a group
# of 128, adapters and none
@pytest.mark.parametrize("name", ["tiny", "decode", "qwen_moe_prefill", "deepseek_v3_slice", "ragged", "no adapters"])
def test_norm_router_and_layer(cuda_device, name):
    """Norm, router product, choice, W8A8 layer: with the norm's 8 bits handed on, y is
    bit-identical to what the layer makes of the norm's bf16 output."""
    if name == "ragged":
        c = custom_case(cuda_device, T=150, K=3, E=5, H=272, I=80, L=4, R=32, ranks=[12, 0, 24, 5], seg_lens=[40, 30, 50, 30],
                        adapters=[0, 3, -1, 2], lora_std="fan_in", seed=2, expert_bias=1.0)
    elif name == "no adapters":
        c = custom_case(cuda_device, T=70, K=2, E=6, H=192, I=256, L=0, R=0, ranks=[], seg_lens=[70], adapters=[-1])
    else:
        c = workload_case(name, cuda_device)
    q, cfg = quant_of(c), c.cfg
    T, H = c.x.shape
    g = torch.Generator().manual_seed(1)
    gain = (1 + 0.1 * torch.randn(H, generator=g)).to(BF).to(cuda_device)
    stream = (3 * torch.randn(T, H, generator=g)).to(BF).to(cuda_device)
    gate = (torch.randn(H, cfg.num_experts, generator=g) / H ** 0.5).to(BF).to(cuda_device)
    codes, exps, y, r = norm.rms_norm_fp8(c.x, gain, 1e-6, stream)
    ids, w = rt.moe_route((y @ gate).float(), cfg.topk, "sigmoid", 0.01 * torch.randn(cfg.num_experts, generator=g).to(cuda_device), check=True)
    want = layer(c, q, y, ids, w)
    assert torch.isfinite(want.float()).all() and want.float().abs().max() > 0
    got = layer(c, q, y, ids, w, x_codes=codes, x_exps=exps)
    assert torch.equal(got, want)
    # the codes are what is multiplied: without adapters y itself is not looked at
    if name == "no adapters":
        assert torch.equal(layer(c, q, torch.zeros_like(y), ids, w, x_codes=codes, x_exps=exps), want)
    else:
        assert not torch.equal(layer(c, q, y, ids, w, x_codes=torch.zeros_like(codes), x_exps=exps), want)


def test_empty_batch_in_8_bits(cuda_device):
    c = workload_case("tiny", cuda_device)
    q = quant_of(c)
    H = c.x.shape[1]
    lo = [getattr(c.w, k) for k in LORA]
    e = lambda *s: torch.empty(*s, dtype=torch.uint8, device=cuda_device)  # noqa: E731
    y = mlr.fused_moe_lora_forward_fp8_w8a8(c.x[:0], c.b.topk_ids[:0], c.b.topk_weights[:0],
                                            torch.zeros(0, dtype=torch.int32, device=cuda_device), c.b.lora_ranks, c.scal,
                                            q.w_gate_up_q, q.w_gate_up_exp, q.w_down_q, q.w_down_exp, *lo, x_codes=e(0, H),
                                            x_exps=e(0, (H + 127) // 128))
    assert y.shape == (0, H)


def test_a_block_served_from_one_graph(cuda_device):
    """Norm, choice, sort, 4-bit layer captured together and replayed on a padded batch
    of other tokens, against eager calls."""
    T, H, I, E, K = 96, 256, 128, 16, 4
    g = torch.Generator().manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, res = rand(T, H).to(BF).cuda(), rand(T, H).to(BF).cuda()
    gain, gate = torch.ones(H, dtype=BF).cuda(), (rand(H, E) / 16).cuda()
    up = fp4.fp4_quantize((rand(E, 2 * I, H) / 16).cuda(), "mxfp4")
    down = fp4.fp4_quantize((rand(E, H, I) / 11).cuda(), "mxfp4")
    mask = torch.ones(T, dtype=torch.bool, device="cuda")

    def block():
        y, r = norm.rms_norm(x, gain, 1e-6, res)
        ids, w = rt.moe_route(y.float() @ gate, K, token_mask=mask)
        return r, ids, fp4.fp4_moe_forward(y, ids, w, *up, *down, "mxfp4", check=False)

    block()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block()
    x.copy_(rand(T, H).to(BF))
    mask[60:] = False
    x[60:] = float("nan")  # what padding holds does not matter
    graph.replay()
    for a, b in zip(out, block()):
        assert torch.equal(a[:60], b[:60])
    r, ids, y = out
    assert (ids[60:] == -1).all() and not y[60:].any() and torch.isfinite(y.float()).all()


def test_a_block_trained(cuda_device):
    """Norm, router, choice with its loss, sorted rows, weighted sum: gradients of
    everything against the same in 64 bits."""
    T, H, E, K = 60, 64, 12, 3
    g = torch.Generator().manual_seed(0)
    mk = lambda *s: torch.randn(*s, generator=g).cuda().requires_grad_()  # noqa: E731
    x, res, gain, gate, mats = mk(T, H), mk(T, H), mk(H), mk(H, E), mk(E, H, H)
    up = torch.randn(T, H, generator=g).cuda()
    leaves = (x, res, gain, gate, mats)

    y, r = norm.RmsNorm.apply(x, gain, 1e-6, res)
    w, ids, loss, counts = rt.MoeRoute.apply(y @ gate / 8, K, "sigmoid", None, 4, 2, True, 2.5)
    rows, pos, off = pm.MoePermute.apply(y, ids, E)
    first = off.tolist()
    out = torch.cat([rows[first[e]:first[e + 1]] @ mats[e] / 8 for e in range(E)])
    z = pm.MoeUnpermute.apply(out.contiguous(), pos, w) + r
    ((z * up).sum() + 100 * loss).backward()
    got = [t.grad.double() for t in leaves]

    xd, rd, gd, td, md = (t.detach().double().requires_grad_() for t in leaves)
    q = xd + rd
    yd = q * gd / (q.square().mean(1, keepdim=True) + 1e-6).sqrt()
    s = torch.sigmoid(yd @ td / 8)
    chosen = s.gather(1, ids.long())
    wd = 2.5 * chosen / chosen.sum(1, keepdim=True)
    p = s / s.sum(1, keepdim=True)
    cnt = counts[:-1].double()
    ld = E / (K * T * T) * (cnt * p.sum(0)).sum()
    zd = torch.einsum("tk,tkh->th", wd, torch.einsum("th,tkhj->tkj", yd, md[ids.long()] / 8)) + q
    ((zd * up).sum() + 100 * ld).backward()
    assert abs(float(loss.detach()) - float(ld.detach())) < 1e-5
    for a, t in zip(got, (xd, rd, gd, td, md)):
        # products of float32 matrices in between: a few hundred roundings of 2^-24 in a row
        assert float((a - t.grad).norm() / t.grad.norm()) < 1e-4


def test_two_host_threads(cuda_device):
    """The operators called by two threads at once, each on a stream of its own."""
    T, H, E, K = 700, 520, 96, 6
    one = torch.ones(1, device="cuda")

    def inputs(seed):
        g = torch.Generator().manual_seed(seed)
        x, res = (torch.randn(T, H, generator=g).to(BF).cuda() for _ in range(2))
        return x, res, torch.ones(H, dtype=BF, device="cuda"), torch.randn(T, E, generator=g).cuda()

    def block(x, res, gain, l):
        codes, exps, y, r = norm.rms_norm_fp8(x, gain, 1e-6, res)
        ids, w = rt.moe_route(l, K, "sigmoid", None, 8, 4)
        loss, counts = rt.moe_balance_loss(l, ids, "sigmoid")
        dl = rt.moe_route_backward(l, ids, w, counts, one, "sigmoid")
        return codes, exps, y, r, ids, w, loss, counts, dl, *norm.rms_norm_backward(y, r, gain, 1e-6, res)

    sets = [inputs(s) for s in range(2)]
    want = [block(*s) for s in sets]
    torch.cuda.synchronize()
    wrong, failed = [], []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    out = block(*sets[i])
                    torch.cuda.current_stream().synchronize()
                    wrong.extend(n for n, (a, b) in enumerate(zip(out, want[i])) if not torch.equal(a, b))
        except Exception as e:  # noqa: BLE001  an exception of a thread is not the test's
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and not wrong
