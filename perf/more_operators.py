"""Cases of the normalisation and routing operators before the experts, with their plain forms.

Operators (field "op" of a case):

  norm        the residual's addition and a root-mean-square norm, its output also (fmt "fp8")
              in 8 bits with a power-of-two scale per 128 columns, and those 8 bits back to numbers
  norm_train  the same norm without the 8 bits, and the gradients of its inputs and weight
  route       the choice of each token's experts from the router's logits with their
              weights, and (train) the gradient of the logits
  balance     the balance loss over a batch with the tokens per expert, and the
              gradient of the logits

Formulas.  Norm: r = x + residual, rounded to the tensors' type; y = r w / sqrt(mean(r^2)
+ eps), rounded.  In 8 bits: 2^s is a group's scale, s the smallest integer >= -127 with
max|y| <= 448 * 2^s (0 for zeros), and the code the nearest E4M3 value of y / 2^s (ties to
even).  With m = 1 / sqrt(mean(r^2) + eps) and h = dy w: dr = m (h - r m^2 mean(h r)) plus
the gradient that reaches r otherwise; dw = sum over rows of dy r m.

Route: logits that are not finite count as -inf; such experts are never chosen.  An
expert's choice score is its logit, or with a bias (or groups, under "sigmoid") its
sigmoid(logit) + bias.  With groups only the experts of the `topk_groups` best groups
stand to choice; a group's score is its best choice score under softmax, the sum of its
two best under sigmoid.  Ties go to the lowest index.  The weights are softmax(logits) or
sigmoid(logits) of the chosen ones, divided by their sum (renormalize), times `scale`.  A
place that no expert is left for, and those of a masked token, have id -1 and weight 0.

Balance: with N tokens that are not masked, c_e pairs of expert e and the shares p_te =
softmax(logits) or sigmoid(logits) over their sum, loss = E / (K N^2) sum_e c_e sum_t p_te.
"""
import math

import torch

own = False

EPS = 1e-6
GROUP = 128


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one new token of a DeepSeek-V3-like model before its experts: latency only
        {"name": "norm token", "op": "norm", "tokens": 1, "hidden": 7168, "dtype": "bf16", "residual": True, "fmt": "fp8"},
        # a decode batch of a Qwen-MoE-like model: one token of each of 256 requests
        {"name": "norm decode", "op": "norm", "tokens": 256, "hidden": 2048, "dtype": "bf16", "residual": True, "fmt": "fp8"},
        # a DeepSeek-V3-like prefill on its way to experts in 8 bits
        {"name": "norm prefill", "op": "norm", "tokens": 8192, "hidden": 7168, "dtype": "bf16", "residual": True, "fmt": "fp8"},
        # a float32 training step with odd sizes, the first norm of a model (nothing to add)
        {"name": "norm_train ragged", "op": "norm_train", "tokens": 1531, "hidden": 1111, "dtype": "fp32", "residual": False},
        # a DeepSeek-V3-like training batch
        {"name": "norm_train large", "op": "norm_train", "tokens": 8192, "hidden": 7168, "dtype": "bf16", "residual": True},
        # the experts of one new token of a Qwen-MoE-like model: latency only
        {"name": "route token", "op": "route", "tokens": 1, "experts": 128, "topk": 8, "scoring": "softmax", "bias": False, "groups": 1, "topk_groups": 1, "renormalize": True, "dtype": "fp32", "pad": 0.0, "closed": 0, "train": False},
        # a decode batch of a DeepSeek-V3-like model: sigmoid, correction bias, the best 4 of 8 groups
        {"name": "route decode", "op": "route", "tokens": 256, "experts": 256, "topk": 8, "scoring": "sigmoid", "bias": True, "groups": 8, "topk_groups": 4, "renormalize": True, "dtype": "fp32", "pad": 0.0, "closed": 0, "train": False},
        # a DeepSeek-V3-like training batch, padded at its end
        {"name": "route train", "op": "route", "tokens": 8192, "experts": 256, "topk": 8, "scoring": "sigmoid", "bias": True, "groups": 8, "topk_groups": 4, "renormalize": True, "dtype": "fp32", "pad": 0.1, "closed": 0, "train": True},
        # odd sizes, weights that are not renormalised, some experts closed
        {"name": "route ragged", "op": "route", "tokens": 1531, "experts": 60, "topk": 6, "scoring": "softmax", "bias": False, "groups": 1, "topk_groups": 1, "renormalize": False, "dtype": "bf16", "pad": 0.0, "closed": 7, "train": True},
        # the batch of the metadata stress test, a million tokens
        {"name": "route stress", "op": "route", "tokens": 1048576, "experts": 256, "topk": 8, "scoring": "softmax", "bias": False, "groups": 1, "topk_groups": 1, "renormalize": True, "dtype": "fp32", "pad": 0.0, "closed": 0, "train": False},
        # a Qwen-MoE-like training batch
        {"name": "balance", "op": "balance", "tokens": 4096, "experts": 128, "topk": 8, "scoring": "softmax", "dtype": "fp32", "pad": 0.0, "closed": 0},
        # all tokens of a large training step, as the loss takes them together
        {"name": "balance large", "op": "balance", "tokens": 262144, "experts": 256, "topk": 8, "scoring": "sigmoid", "dtype": "fp32", "pad": 0.1, "closed": 0},
    ]


def _spread(rng, low, high, multiple=1):
    """A size between low and high, spread over its logarithm; half of them odd where `multiple` is 1."""
    v = int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))
    v = max(low, min(high, v))
    if multiple > 1:
        return max(multiple, v // multiple * multiple)
    return min(high, v | 1) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_train", "route", "route", "balance"])
    if op in ("norm", "norm_train"):
        hidden = _spread(rng, 64, 16384, rng.choice([1, 8, 128]))
        case = {"op": op, "hidden": hidden, "tokens": _spread(rng, 1, max(1, 8192 * 7168 // 2 // hidden)),
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "residual": rng.random() < 0.75}
        return case | {"fmt": rng.choice(["none", "fp8"])} if op == "norm" else case
    experts = _spread(rng, 2, 512, rng.choice([1, 8, 32]))
    topk = rng.randint(1, min(16, max(1, experts // 2)))
    case = {"op": op, "experts": experts, "topk": topk, "tokens": _spread(rng, 1, min(1048576, 33554432 // experts)),
            "scoring": rng.choice(["softmax", "sigmoid"]), "dtype": rng.choice(["fp32", "fp32", "bf16"]),
            "pad": rng.choice([0.0, 0.0, 0.2]), "closed": rng.choice([0, 0, experts // 8])}
    if op == "route":
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0])
        best = rng.randint(max(1, -(-topk * groups // experts)), groups)
        case |= {"groups": groups, "topk_groups": best, "bias": case["scoring"] == "sigmoid" and rng.random() < 0.7,
                 "renormalize": topk > 1 and rng.random() < 0.7, "train": rng.random() < 0.5}
    return case


def work(case):
    T, s = case["tokens"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_train"):
        H, ways = case["hidden"], 2 if case["residual"] else 1
        forward = 2 * ways * T * H * s  # x, residual -> y, r
        if case["op"] == "norm":  # then codes and scales, and the numbers back from them
            eight = (2 * (T * H + T * -(-H // GROUP)) + 2 * T * H) if case["fmt"] == "fp8" else 0
            return {"bytes": forward + eight + H * s, "flops": 8 * T * H}
        return {"bytes": forward + (2 + ways) * T * H * s + H * (s + 4), "flops": 16 * T * H}  # dy, r, the other gradient of r -> dr, dw
    E, K = case["experts"], case["topk"]
    if case["op"] == "route":
        forward = T * E * s + 8 * T * K
        if not case["train"]:
            return {"bytes": forward, "flops": 4 * T * E}
        # renormalised weights need only the chosen logits again
        again = T * E * s if not case["renormalize"] and case["scoring"] == "softmax" else T * K * s
        return {"bytes": forward + again + 8 * T * K + T * E * s, "flops": 8 * T * E}
    return {"bytes": 3 * T * E * s + 4 * T * K + 4 * (E + 2), "flops": 14 * T * E}  # logits, ids -> loss, counts; logits -> their gradient


# ----------------------------------------------------------------- inputs --
def _dtype(case):
    return torch.float32 if case["dtype"] == "fp32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, T = _dtype(case), case["tokens"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    state = {k: case.get(k) for k in ("op", "fmt", "topk", "scoring", "groups", "topk_groups", "renormalize", "train")}
    if case["op"] in ("norm", "norm_train"):
        H = case["hidden"]
        state["x"] = normal(T, H).to(dt)
        # the residual stream of a deep model: larger than what a layer adds, some columns far larger
        state["residual"] = (2 * normal(T, H) * (1 + 8 * (torch.rand(H, generator=g, device="cuda") < 0.01))).to(dt) if case["residual"] else None
        state["w"] = (1 + 0.2 * normal(H)).to(dt)
        if case["op"] == "norm_train":
            state["dy"] = normal(T, H).to(dt)
            state["dr"] = normal(T, H).to(dt) if case["residual"] else None
        return state
    E, K = case["experts"], case["topk"]
    logits = normal(T, E) + 0.5 * normal(E)  # a router with uneven experts
    if case["closed"]:
        logits[:, torch.randperm(E, generator=g, device="cuda")[: case["closed"]]] = -math.inf
    state["logits"] = logits.to(dt)
    pad = int(T * case["pad"])
    state["mask"] = torch.arange(T, device="cuda") < T - pad if pad else None
    if case["op"] == "route":
        state["bias"] = 0.05 * normal(E) if case["bias"] else None
        state["scale"] = 2.5 if case["scoring"] == "sigmoid" else 1.0
        if case["train"]:
            state["d_weights"] = normal(T, K)
        return state
    state["ids"] = _choose(state["logits"], K, "softmax", None, 1, 1, state["mask"])
    state["d_loss"] = torch.full((1,), 0.01, device="cuda")  # the loss's coefficient
    return state


# ------------------------------------------------------------ plain forms --
def _norm(x, residual, w):
    r = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    f = r.float()
    m = 1 / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)
    return (f * m * w.float()).to(x.dtype), r


def _groups_of(v):
    """Columns [T, H] in groups [T, groups, 128], zeros past H."""
    return torch.nn.functional.pad(v, (0, -v.shape[-1] % GROUP)).unflatten(-1, (-1, GROUP))


def _eight_bits(y):
    """The numbers that y [T, H] stands for after its rounding to 8 bits."""
    b = _groups_of(y.float())
    most = b.abs().amax(-1, keepdim=True)
    part, power = torch.frexp(most)  # most = part 2^power, part in [0.5, 1): 448 * 2^s = 0.875 * 2^(s + 9)
    s = torch.where(most > 0, (power - 9 + (part > 0.875).int()).clamp(min=-127), 0).int()
    up, down = ((127 - s) << 23).view(torch.float32), torch.ldexp(torch.ones_like(most), s)
    codes = (b * up).to(torch.float8_e4m3fn)
    return (codes.float() * down).flatten(-2)[..., : y.shape[-1]].bfloat16()  # which holds an E4M3 value and a power of two


def _norm_gradients(dy, dr, r, w):
    f, h = r.float(), dy.float() * w.float()
    m = 1 / torch.sqrt((f * f).mean(-1, keepdim=True) + EPS)
    dx = m * (h - f * m * m * (h * f).mean(-1, keepdim=True))
    return (dx if dr is None else dx + dr.float()).to(r.dtype), (dy.float() * f * m).sum(0)


def _finite(logits, dtype=torch.float32):
    v = logits.to(dtype)
    return torch.where(torch.isfinite(v), v, -math.inf)


def _choose(logits, K, scoring, bias, groups, best, mask):
    """Ids int32 [T, K] of the experts chosen for each token, -1 where none is left."""
    score = _finite(logits)
    if scoring == "sigmoid" and (bias is not None or groups > 1):
        score = score.double()  # two scores may be nearer to one another than 32 bits tell
        score = torch.where(score == -math.inf, score, 1 / (1 + torch.exp(-score)) + (0.0 if bias is None else bias.double()))
    if groups > 1:
        parts = score.unflatten(-1, (groups, -1)).sort(-1, descending=True).values
        value = parts[..., 0]
        if scoring == "sigmoid" and parts.shape[-1] > 1:
            value = value + torch.where(parts[..., 1] == -math.inf, 0.0, parts[..., 1])
        order = value.sort(stable=True, dim=-1, descending=True).indices
        out = torch.ones_like(value, dtype=torch.bool).scatter(-1, order[:, :best], False)
        score = torch.where(out.repeat_interleave(parts.shape[-1], -1), -math.inf, score)
    by, ids = score.sort(stable=True, dim=-1, descending=True)
    by, ids = by[:, :K], ids[:, :K]
    left = by > -math.inf if mask is None else (by > -math.inf) & mask[:, None]
    return torch.where(left, ids, -1).int()


def _scores(logits, scoring):
    """softmax or sigmoid of all logits, zeros in rows and places without finite ones."""
    v = _finite(logits)
    if scoring == "sigmoid":
        return 1 / (1 + torch.exp(-v))
    most = v.amax(-1, keepdim=True)
    e = torch.exp(v - torch.where(most == -math.inf, 0.0, most))
    return torch.where(most == -math.inf, 0.0, e / e.sum(-1, keepdim=True))


def _weights(logits, ids, scoring, renormalize, scale):
    """The chosen experts' scores [T, K] (0 where none is), their divisor, and the weights."""
    at = ids.clamp(min=0).long()
    if renormalize and scoring == "softmax":
        v = torch.where(ids < 0, -math.inf, _finite(logits.gather(-1, at)))
        most = v.amax(-1, keepdim=True)
        s = torch.exp(v - torch.where(most == -math.inf, 0.0, most))
    else:
        s = torch.where(ids < 0, 0.0, _scores(logits, scoring).gather(-1, at))
    total = s.sum(-1, keepdim=True) if renormalize else torch.ones_like(s[:, :1])
    return s, total, torch.where(total > 0, s / total, 0.0) * scale


def _route_gradient(d_weights, logits, ids, scoring, renormalize, scale):
    s, total, w = _weights(logits, ids, scoring, renormalize, scale)
    g = torch.where(ids < 0, 0.0, d_weights)
    if scoring == "sigmoid":
        ds = (g * scale - (g * w).sum(-1, keepdim=True)) / total if renormalize else g * scale
        d = torch.where(total > 0, ds * s * (1 - s), 0.0)
    else:
        d = g * w - (w / scale * (g * w).sum(-1, keepdim=True) if renormalize else 0.0)
    out = torch.zeros(logits.shape[0], logits.shape[1] + 1, device=logits.device)
    out.scatter_(-1, torch.where(ids < 0, logits.shape[1], ids).long(), d)
    out = out[:, :-1]
    if scoring == "softmax" and not renormalize:
        out = out - _scores(logits, scoring) * (g * w).sum(-1, keepdim=True)
    return out.to(logits.dtype)


def _shares(logits, scoring, mask):
    s = _scores(logits, scoring)
    total = s.sum(-1, keepdim=True)
    p = s if scoring == "softmax" else torch.where(total > 0, s / total, 0.0)
    return s, p if mask is None else torch.where(mask[:, None], p, 0.0)


def _plain(state):
    op = state["op"]
    if op == "norm":
        y, r = _norm(state["x"], state["residual"], state["w"])
        return {"y": y, "r": r, "values": _eight_bits(y) if state["fmt"] == "fp8" else None}
    if op == "norm_train":
        y, r = _norm(state["x"], state["residual"], state["w"])
        dx, dw = _norm_gradients(state["dy"], state["dr"], r, state["w"])
        return {"y": y, "r": r, "dx": dx, "dw": dw}
    logits, scoring, mask, K = state["logits"], state["scoring"], state["mask"], state["topk"]
    T, E = logits.shape
    if op == "route":
        ids = _choose(logits, K, scoring, state["bias"], state["groups"], state["topk_groups"], mask)
        out = {"ids": ids, "weights": _weights(logits, ids, scoring, state["renormalize"], state["scale"])[2]}
        if state["train"]:
            out["d_logits"] = _route_gradient(state["d_weights"], logits, ids, scoring, state["renormalize"], state["scale"])
        return out
    ids = state["ids"]
    held = (ids >= 0) & (ids < E) if mask is None else (ids >= 0) & (ids < E) & mask[:, None]
    counts = torch.bincount(torch.where(held, ids, E).reshape(-1), minlength=E + 1)[:E]
    n = torch.full((), float(T), dtype=torch.float64, device="cuda") if mask is None else mask.sum().double()
    s, p = _shares(logits, scoring, mask)
    a = counts.double() * (E / K) / (n * n).clamp(min=1)
    loss = (a * p.sum(0, dtype=torch.float64)).sum().float()
    a = (a * state["d_loss"]).float()
    d = p * (a - (p * a).sum(-1, keepdim=True))
    return {"loss": loss, "counts": torch.cat((counts, n.long().reshape(1))).int(),
            "d_logits": (d if scoring == "softmax" else d * (1 - s)).to(logits.dtype)}


def run(state):
    if not own:
        return _plain(state)
    from lora_moe_expert_info_gb300 import norm, router
    op = state["op"]
    if op == "norm" and state["fmt"] == "fp8":
        codes, exps, y, r = norm.rms_norm_fp8(state["x"], state["w"], EPS, state["residual"])
        return {"y": y, "r": r, "values": norm.fp8_dequantize(codes, exps)}
    if op in ("norm", "norm_train"):
        y, r = norm.rms_norm(state["x"], state["w"], EPS, state["residual"])
        if op == "norm":
            return {"y": y, "r": r, "values": None}
        dx, dw = norm.rms_norm_backward(state["dy"], r, state["w"], EPS, state["dr"])
        return {"y": y, "r": r, "dx": dx, "dw": dw}
    logits, scoring, mask, K = state["logits"], state["scoring"], state["mask"], state["topk"]
    if op == "route":
        ids, weights = router.moe_route(logits, K, scoring, state["bias"], state["groups"], state["topk_groups"],
                                        state["renormalize"], state["scale"], token_mask=mask)
        out = {"ids": ids, "weights": weights}
        if state["train"]:
            out["d_logits"] = router.moe_route_backward(logits, ids, state["d_weights"], scoring=scoring,
                                                        renormalize=state["renormalize"], scale=state["scale"])
        return out
    loss, counts = router.moe_balance_loss(logits, state["ids"], scoring, token_mask=mask)
    d = router.moe_route_backward(logits, state["ids"], counts=counts, d_loss=state["d_loss"], scoring=scoring, token_mask=mask)
    return {"loss": loss, "counts": counts, "d_logits": d}


# ------------------------------------------------------------- definition --
def exact(case, seed):
    state = prepare(case, seed)
    dt = _dtype(case)
    if case["op"] in ("norm", "norm_train"):
        H = case["hidden"]
        r = state["x"].double() if state["residual"] is None else state["x"].double() + state["residual"].double()
        q = r.to(dt).double()
        w = state["w"].double()
        rms = torch.sqrt(torch.einsum("th,th->t", q, q) / H + EPS)[:, None]
        y = q / rms * w
        if case["op"] == "norm":
            values = None
            if case["fmt"] == "fp8":
                v = y.to(dt).double()
                values = torch.empty_like(v)
                for c in range(0, H, GROUP):
                    b = v[:, c:c + GROUP]
                    most = b.abs().amax(1, keepdim=True)
                    s = torch.where(most > 0, torch.ceil(torch.log2(most / 448)).clamp(min=-127), 0.0)
                    a = b * torch.exp2(-s)
                    # E4M3: four significant bits down to 2^-6, steps of 2^-9 below
                    step = torch.exp2(torch.floor(torch.log2(a.abs().clamp(min=2.0 ** -6))) - 3)
                    values[:, c:c + GROUP] = torch.round(a / step) * step * torch.exp2(s)
            return {"y": y, "r": r, "values": values}
        # the gradient of sum(y dy) as a product with the Jacobian: dy_i/dr_j = w_i ((i = j) - r_i r_j / (H rms^2)) / rms
        g = state["dy"].double()
        dot = torch.einsum("th,h,th->t", g, w, q)[:, None]
        dx = (g * w - q * dot / (H * rms ** 2)) / rms
        if state["dr"] is not None:
            dx = dx + state["dr"].double()
        return {"y": y, "r": r, "dx": dx, "dw": torch.einsum("th,th->h", g, q / rms)}
    T, E, K = case["tokens"], case["experts"], case["topk"]
    l = state["logits"].double()
    open_ = torch.isfinite(l)
    if case["scoring"] == "softmax":
        z = torch.where(open_, l, -math.inf)
        s = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
        s = torch.where(open_, s, 0.0)
    else:
        s = torch.where(open_, torch.sigmoid(l), 0.0)
    kept = torch.ones(T, dtype=torch.bool, device="cuda") if state["mask"] is None else state["mask"]
    if case["op"] == "route":
        taken = torch.zeros(T, E, dtype=torch.bool, device="cuda")
        score = torch.where(open_, l, -math.inf)
        if case["scoring"] == "sigmoid" and (case["bias"] or case["groups"] > 1):
            score = torch.where(open_, torch.sigmoid(l) + (state["bias"].double() if case["bias"] else 0.0), -math.inf)
        if case["groups"] > 1:
            size = E // case["groups"]
            top = score.view(T, -1, size).topk(min(size, 2 if case["scoring"] == "sigmoid" else 1), -1).values
            value = torch.where(top[..., :1].isfinite(), torch.where(top.isfinite(), top, 0.0).sum(-1, keepdim=True), -math.inf)[..., 0]
            for _ in range(case["groups"] - case["topk_groups"]):  # the worst group leaves; of equal ones the last
                worst = value.shape[1] - 1 - value.flip(1).argmin(1)
                value[torch.arange(T), worst] = math.inf
                score.view(T, -1, size)[torch.arange(T), worst] = -math.inf
        weights = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        ids = torch.zeros(T, K, dtype=torch.long, device="cuda")
        for k in range(K):  # one expert after another, the first of the best
            best = score.max(1)
            ids[:, k] = best.indices
            good = kept & (best.values > -math.inf)
            weights[:, k] = torch.where(good, s.gather(1, best.indices[:, None])[:, 0], 0.0)
            taken[torch.arange(T), best.indices] |= good
            score.scatter_(1, best.indices[:, None], -math.inf)
        total = weights.sum(1, keepdim=True)
        c = state["scale"]
        w = c * weights / torch.where(total > 0, total, 1.0) if case["renormalize"] else c * weights
        out = {"ids": None, "weights": w}
        if case["train"]:
            g = torch.zeros(T, E, dtype=torch.float64, device="cuda")
            for k in range(K):
                g.scatter_add_(1, ids[:, k:k + 1], torch.where(weights[:, k:k + 1] > 0, state["d_weights"][:, k:k + 1].double(), 0.0))
            u = torch.where(taken, s, 0.0)
            if case["renormalize"]:  # w = c u / sum(u)
                total = torch.where(total > 0, total, 1.0)
                g = torch.where(taken, (g - (g * u).sum(1, keepdim=True) / total) / total, 0.0)
            gs = c * g
            out["d_logits"] = gs * s * (1 - s) if case["scoring"] == "sigmoid" else s * (gs - (gs * s).sum(1, keepdim=True))
        return out
    n = float(kept.sum())
    ids = state["ids"].long()
    counts = torch.stack([((ids == e) & kept[:, None]).sum() for e in range(E)]).double()
    total = s.sum(1, keepdim=True)
    p = torch.where(kept[:, None] & (total > 0), s / torch.where(total > 0, total, 1.0), 0.0)
    a = E * counts / (K * max(n, 1.0) ** 2)
    loss = torch.einsum("te,e->", p, a)
    h = state["d_loss"].double() * a
    d = p * (h - (p @ h)[:, None])
    return {"loss": loss, "counts": None, "d_logits": d if case["scoring"] == "softmax" else d * (1 - s)}
