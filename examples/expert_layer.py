"""An expert layer trained through the sorted rows, then served from 4-bit experts.

Training: each token's experts are chosen (MoeRoute), tokens sorted by expert
(MoePermute), every expert's rows go
through its frozen weights plus trainable low-rank adapters with plain matrix
products, and the rows are weighted and summed back (MoeUnpermute); gradients
reach the adapters, the router and the tokens.  Serving: the adapters are merged,
the experts quantised once (fp4_quantize), and moe_route and fp4_moe_forward answer
a prompt and single tokens from them.

    python examples/expert_layer.py [--steps 20] [--fmt nvfp4]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from lora_moe_expert_info_gb300 import fp4  # noqa: E402
from lora_moe_expert_info_gb300.permute import MoePermute, MoeUnpermute  # noqa: E402
from lora_moe_expert_info_gb300.router import MoeRoute, moe_route  # noqa: E402


def route(x, router, topk):
    """Expert ids int32 [T, K] and renormalised weights float32 [T, K], with gradients."""
    weights, ids, _, _ = MoeRoute.apply(x.float() @ router, topk)
    return ids, weights


class ExpertLayer(torch.nn.Module):
    """y_t = sum_k w[t,k] W_down,e [SiLU(W_gate,e x_t) * (W_up,e x_t)], W = frozen + B A."""

    def __init__(self, experts, topk, hidden, intermediate, rank, seed=0):
        super().__init__()
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g) * std).cuda().bfloat16()

        self.topk = topk
        self.w_gate_up = normal(experts, 2 * intermediate, hidden, std=1 / math.sqrt(hidden))
        self.w_down = normal(experts, hidden, intermediate, std=1 / math.sqrt(intermediate))
        self.router = torch.nn.Parameter(normal(hidden, experts, std=1 / math.sqrt(hidden)).float())
        self.a_gate_up = torch.nn.Parameter(normal(experts, rank, hidden, std=1 / math.sqrt(hidden)).float())
        self.b_gate_up = torch.nn.Parameter(torch.zeros(experts, 2 * intermediate, rank, device="cuda"))
        self.a_down = torch.nn.Parameter(normal(experts, rank, intermediate, std=1 / math.sqrt(intermediate)).float())
        self.b_down = torch.nn.Parameter(torch.zeros(experts, hidden, rank, device="cuda"))

    def merged(self):
        """The experts' matrices with their adapters, float32."""
        return self.w_gate_up + self.b_gate_up @ self.a_gate_up, self.w_down + self.b_down @ self.a_down

    def forward(self, x):
        ids, weights = route(x, self.router, self.topk)
        rows, pair_pos, offsets = MoePermute.apply(x, ids, self.router.shape[1])
        gate_up, down = (w.to(x.dtype) for w in self.merged())
        first = offsets.tolist()
        out = []
        for e in range(gate_up.shape[0]):
            g, u = (rows[first[e]:first[e + 1]] @ gate_up[e].T).chunk(2, -1)
            out.append((torch.nn.functional.silu(g) * u) @ down[e].T)
        out.append(rows[first[-1]:])  # rows of masked pairs: zeros
        return MoeUnpermute.apply(torch.cat(out).contiguous(), pair_pos, weights)


class QuantisedExperts:
    """The layer's experts in 4 bits, for serving."""

    def __init__(self, layer, fmt, calibration):
        self.layer, self.fmt = layer, fmt
        self.matrices, self.scales = [], []
        for w in layer.merged():
            w = w.detach().contiguous()
            scale = w.abs().amax((1, 2)) / 2688 if fmt == "nvfp4" else None
            self.matrices += fp4.fp4_quantize(w, fmt, scale)
            self.scales.append(scale)
        # the activations' tensor scales, fixed from a calibration batch
        self.x_scale = calibration.abs().max().float().reshape(1) / 2688 if fmt == "nvfp4" else None
        self.h_scale = torch.full((1,), 32 / 2688, device="cuda") if fmt == "nvfp4" else None

    @torch.no_grad()
    def __call__(self, x):
        ids, weights = moe_route(x.float() @ self.layer.router, self.layer.topk)
        return fp4.fp4_moe_forward(x, ids, weights, *self.matrices, self.fmt, *self.scales, self.x_scale, self.h_scale)


def run(steps=20, fmt="nvfp4", experts=8, topk=2, hidden=256, intermediate=512, rank=8, tokens=512, seed=0):
    """Trains towards a teacher layer; returns the losses and the relative error
    of the 4-bit answers to a prompt and to its last token alone."""
    layer = ExpertLayer(experts, topk, hidden, intermediate, rank, seed)
    x = torch.randn(tokens, hidden, generator=torch.Generator().manual_seed(seed + 1)).cuda().bfloat16()
    with torch.no_grad():
        target = 1.5 * layer(x)
    opt = torch.optim.Adam(layer.parameters(), lr=2e-3)
    losses = []
    for _ in range(steps):
        loss = (layer(x).float() - target.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    served = QuantisedExperts(layer, fmt, x)
    with torch.no_grad():
        want = layer(x).float()
    prompt, token = served(x).float(), served(x[-1:].contiguous()).float()
    return losses, float((prompt - want).norm() / want.norm()), float((token - want[-1:]).norm() / want[-1:].norm())


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--fmt", choices=sorted(fp4.FORMATS), default="nvfp4")
    a = ap.parse_args()
    losses, prompt, token = run(a.steps, a.fmt)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    print(f"4-bit experts ({a.fmt}): relative error {prompt:.3f} on the prompt, {token:.3f} on one token")
