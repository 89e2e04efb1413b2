"""Cases of the expert-sorting and 4-bit floating-point operators, with their plain forms.

Operators (field "op" of a case):

  permute    tokens copied into rows sorted by expert, and the gradient of the copy
  unpermute  the rows weighted and summed back per token, and the gradients of
             rows and weights
  quantize   tokens to microscaled 4-bit floats (MXFP4 or NVFP4), sorted by
             expert on the way (topk 0: row by row), and back to numbers
  swiglu     sorted rows [gate | up] to the 4-bit codes of u * SiLU(g), and back
             to numbers
  product    sorted 4-bit rows times their expert's 4-bit weight matrix

Formulas.  A pair p = t*K + k is token t's k-th choice.  Pairs are sorted by
expert id, stable in p; a pair whose id is not in [0, E) comes last, its row is
zero and its place is given as ~row.  MXFP4: blocks of 32 with scale 2^s, s the
smallest integer in [-127, 127] with max|x| <= 6 * 2^s (0 for a block of zeros).
NVFP4: blocks of 16 with an E4M3 scale, the rounded min(max|x| / (6 g), 448), for
a float32 tensor scale g.  A code is x divided by its scale, rounded to the
nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code), sign kept.  Block
scales lie in 512-byte atoms of 128 rows by 4 blocks: row r of the atom, block c
at byte 16 (r mod 32) + 4 (r div 32) + c; the rows of expert e begin at atom row
block offsets[e] div 128 + e.
"""
import math

import torch

own = False

TABLE = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
FLOAT_MAX = 3.4028234663852886e38


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # one new token of a Qwen-MoE-like model on its way to 8 of 128 experts: latency only
        {"name": "permute token", "op": "permute", "tokens": 1, "topk": 8, "experts": 128, "hidden": 2048, "dtype": "bf16", "drop": 0.0},
        # a DeepSeek-V3-like prefill or training batch: 0.9 GB of sorted rows
        {"name": "permute prefill", "op": "permute", "tokens": 8192, "topk": 8, "experts": 256, "hidden": 7168, "dtype": "bf16", "drop": 0.0},
        # a float32 training step with odd sizes and masked pairs
        {"name": "unpermute ragged", "op": "unpermute", "tokens": 1531, "topk": 6, "experts": 60, "hidden": 1111, "dtype": "fp32", "drop": 0.1},
        # a Qwen-MoE-like training batch
        {"name": "unpermute prefill", "op": "unpermute", "tokens": 4096, "topk": 8, "experts": 128, "hidden": 2048, "dtype": "bf16", "drop": 0.0},
        # a decode batch: one token of each of 256 requests
        {"name": "quantize decode", "op": "quantize", "tokens": 256, "topk": 8, "experts": 128, "hidden": 2048, "dtype": "bf16", "drop": 0.0, "fmt": "nvfp4"},
        # a DeepSeek-V3-like prefill
        {"name": "quantize prefill", "op": "quantize", "tokens": 8192, "topk": 8, "experts": 256, "hidden": 7168, "dtype": "bf16", "drop": 0.0, "fmt": "mxfp4"},
        # few rows, sizes that end inside blocks and atoms
        {"name": "swiglu ragged", "op": "swiglu", "tokens": 389, "topk": 2, "experts": 16, "hidden": 1416, "dtype": "bf16", "drop": 0.05, "fmt": "mxfp4"},
        # the hidden activations of a Qwen-MoE-like prefill
        {"name": "swiglu prefill", "op": "swiglu", "tokens": 4096, "topk": 8, "experts": 128, "hidden": 768, "dtype": "bf16", "drop": 0.0, "fmt": "nvfp4"},
        # one token through the gate and up matrices of its 8 experts: reads weights, nothing else
        {"name": "product token", "op": "product", "tokens": 1, "topk": 8, "experts": 128, "hidden": 2048, "outputs": 1536, "drop": 0.0, "fmt": "nvfp4"},
        # a decode batch through the down matrices
        {"name": "product decode", "op": "product", "tokens": 256, "topk": 8, "experts": 128, "hidden": 768, "outputs": 2048, "drop": 0.0, "fmt": "mxfp4"},
        # a Qwen-MoE-like prefill through the gate and up matrices
        {"name": "product prefill", "op": "product", "tokens": 4096, "topk": 8, "experts": 128, "hidden": 2048, "outputs": 1536, "drop": 0.0, "fmt": "nvfp4"},
        # an eighth of a DeepSeek-V3-like prefill through the gate and up matrices
        {"name": "product large", "op": "product", "tokens": 1024, "topk": 8, "experts": 32, "hidden": 7168, "outputs": 4096, "drop": 0.0, "fmt": "mxfp4"},
    ]


def _spread(rng, low, high, multiple=1):
    """A size between low and high, spread over its logarithm; half of them odd multiples."""
    v = int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))
    v = max(low, min(high, v))
    if multiple > 1:
        v = max(multiple, v // multiple * multiple)
    elif rng.random() < 0.5:
        v |= 1
    v = min(v, high)
    return v - multiple if v == 3072 else v


def draw(rng):
    op = rng.choice(["permute", "unpermute", "quantize", "swiglu", "product", "product"])
    experts = _spread(rng, 1, 256)
    topk = rng.randint(1, min(8, experts))
    case = {"op": op, "experts": experts, "topk": topk, "drop": rng.choice([0.0, 0.0, 0.1])}
    if op == "product":
        hidden = _spread(rng, 64, 7168, rng.choice([1, 32, 64]))
        most = 32 * 4096 * 7168  # the weights of the largest listed case
        outputs = _spread(rng, 64, 4096, rng.choice([1, 8, 128]))
        experts = case["experts"] = max(topk, min(experts, most // (hidden * outputs)))
        tokens = _spread(rng, 1, max(1, min(4096, 1024 * 8 * 4096 * 7168 // (topk * hidden * outputs))))
        case.update(tokens=tokens, hidden=hidden, outputs=outputs)
    else:
        hidden = _spread(rng, 64, 7168, rng.choice([1, 8, 64]))
        case.update(tokens=_spread(rng, 1, max(1, min(16384, 8192 * 8 * 7168 // (topk * hidden) // 2))), hidden=hidden)
        case["dtype"] = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("quantize", "swiglu", "product"):
        case["fmt"] = rng.choice(["nvfp4", "mxfp4"])
    if case["tokens"] * topk == 3072 or (op == "swiglu" and 2 * case["hidden"] == 3072):
        case.update(tokens=case["tokens"] + 1, hidden=case["hidden"] - 32)
    if op == "quantize" and rng.random() < 0.25:
        case.update(topk=0, experts=1, drop=0.0)  # a matrix row by row, as weights are quantised
    return case


def _rows(case):
    return case["tokens"] * max(1, case["topk"])


def work(case):
    op, T, E, H = case["op"], case["tokens"], case["experts"], case["hidden"]
    P, s = _rows(case), 2 if case.get("dtype", "bf16") == "bf16" else 4
    if op == "permute":  # x, ids -> rows, places, offsets; row gradients -> token gradients
        return {"bytes": 2 * (T + P) * H * s + 12 * P + 4 * (E + 1), "flops": P * H}
    if op == "unpermute":  # rows, weights -> y; dy, rows -> row and weight gradients
        return {"bytes": (2 * P + 2 * T + P) * H * s + 20 * P, "flops": 5 * P * H}
    if op == "quantize":  # x -> codes and scales -> bf16
        block = 16 if case["fmt"] == "nvfp4" else 32
        return {"bytes": T * H * s + P * (H + 2 * H / block) + 2 * P * H, "flops": 4 * T * H + 2 * P * H}
    if op == "swiglu":
        block = 16 if case["fmt"] == "nvfp4" else 32
        return {"bytes": 2 * P * H * s + P * (H + 2 * H / block) + 2 * P * H, "flops": 12 * P * H}
    block, N = 16 if case["fmt"] == "nvfp4" else 32, case["outputs"]
    used = E if P >= 8 * E else E * (1 - (1 - 1 / E) ** P)  # experts that get a row
    used = max(used, min(E, case["topk"]))
    return {"bytes": (used * N + P) * H * (0.5 + 1 / block) + 2 * P * N, "flops": 2 * P * N * H}


# ----------------------------------------------------------------- inputs --
def _dtype(case):
    return torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16


def _routing(case, g):
    """Expert ids [T, K] of a router with uneven experts, masked pairs at -1, and the weights."""
    T, K, E = case["tokens"], case["topk"], case["experts"]
    bias = 0.5 * torch.randn(E, generator=g, device="cuda")
    logits = torch.randn(T, E, generator=g, device="cuda") + bias
    top = logits.softmax(-1).topk(K, dim=-1)
    ids = top.indices.int()
    weights = top.values / top.values.sum(-1, keepdim=True)
    if case["drop"]:
        ids = torch.where(torch.rand(T, K, generator=g, device="cuda") < case["drop"], -1, ids)
    return ids.int().contiguous(), weights.float().contiguous()


def _pack(q):
    """Code numbers [..., C] to bytes [..., 16 ceil(C / 32)], even column in the low half."""
    C = q.shape[-1]
    q = torch.nn.functional.pad(q, (0, -C % 32)).to(torch.uint8)
    return (q[..., 0::2] | (q[..., 1::2] << 4)).contiguous()


def _atoms(s, block_row, row, blocks):
    """Scale bytes s [R, n] laid out in atoms: row i goes to row `row[i]` of row block `block_row[i]`."""
    n = s.shape[1]
    groups = -(-n // 4)
    s = torch.nn.functional.pad(s, (0, groups * 4 - n)).reshape(-1, groups, 4)
    out = torch.zeros(blocks, groups, 32, 4, 4, dtype=torch.uint8, device=s.device)
    out[block_row, :, row % 32, row // 32] = s
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, T, K, E, H, P = case["op"], case["tokens"], case["topk"], case["experts"], case["hidden"], _rows(case)
    dt = _dtype(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    state = {"op": op, "experts": E, "topk": K, "fmt": case.get("fmt"), "cols": H}
    if K:
        state["ids"], state["weights"] = _routing(case, g)
    if op == "permute":
        return state | {"x": normal(T, H).to(dt), "d_rows": normal(P, H).to(dt)}
    pos, offsets = _sort(state["ids"], E) if K else (None, None)
    state |= {"pos": pos, "offsets": offsets}
    if op == "unpermute":
        return state | {"rows": normal(P, H).to(dt), "dy": normal(T, H).to(dt)}
    if op == "quantize":
        x = normal(T, H).to(dt)
        return state | {"x": x, "scale": x.abs().max().float().reshape(1) / 2688 if case["fmt"] == "nvfp4" else None}
    if op == "swiglu":
        # a calibrated tensor scale, as a server keeps it: |h| stays below 24
        return state | {"x": normal(P, 2 * H).to(dt), "scale": torch.full((1,), 24 / 2688, device="cuda") if case["fmt"] == "nvfp4" else None}
    N = case["outputs"]
    a, w = normal(P, H), normal(E, N, H) / math.sqrt(H)
    nv = case["fmt"] == "nvfp4"
    ga = a.abs().max().reshape(1) / 2688 if nv else None
    gw = w.abs().amax((1, 2)) / 2688 if nv else None
    qa, sa = _quantize(a, case["fmt"], ga)
    qw, sw = _quantize(w, case["fmt"], None if gw is None else gw[:, None, None])
    i = torch.arange(P, device="cuda")
    e = _expert_of(offsets, i, E)
    j = i - offsets[e].long()
    n = torch.arange(N, device="cuda").repeat(E)
    be = torch.arange(E, device="cuda").repeat_interleave(N) * (-(-N // 128))
    return state | {
        "a_codes": _pack(qa), "a_scales": _atoms(sa, offsets[e].long() // 128 + e + j // 128, j % 128, P // 128 + E),
        "w_codes": _pack(qw), "w_scales": _atoms(sw.flatten(0, 1), be + n // 128, n % 128, E * (-(-N // 128))).unflatten(0, (E, -1)),
        "a_scale": ga, "w_scale": gw, "most": max(1, int((offsets[1:] - offsets[:-1]).max())),
    }


# ------------------------------------------------------------ plain forms --
def _sort(ids, E):
    """Places of the pairs [T, K] and the experts' first rows [E + 1], int32."""
    key = ids.reshape(-1).long()
    key = torch.where((key >= 0) & (key < E), key, E)
    by, order = key.sort(stable=True)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=ids.device)
    offsets = torch.searchsorted(by, torch.arange(E + 1, device=ids.device))
    return torch.where(key < E, pos, ~pos).int().reshape(ids.shape), offsets.int()


def _expert_of(offsets, i, E):
    """The expert of each sorted row (E - 1 for a row past the last one)."""
    return (torch.searchsorted(offsets, i.int(), right=True) - 1).clamp(0, E - 1)


def _take(rows, pos):
    """The rows [T, K, H] of the pairs in float32, zeros for masked pairs."""
    at = torch.where(pos < 0, ~pos, pos).long()
    return torch.where((pos < 0)[..., None], 0.0, rows[at].float())


def _put(values, pos):
    """The pairs' values [T, K, H] in sorted rows [P, H], zeros for masked pairs."""
    at = torch.where(pos < 0, ~pos, pos).long().reshape(-1)
    out = torch.empty(at.numel(), values.shape[-1], dtype=values.dtype, device=values.device)
    out[at] = torch.where((pos < 0)[..., None], 0.0, values).reshape(at.numel(), -1).to(values.dtype)
    return out


def _quantize(v, fmt, scale):
    """Float32 values [..., C] to code numbers (0 to 15) [..., C] and scale bytes [..., blocks]."""
    block = 16 if fmt == "nvfp4" else 32
    C = v.shape[-1]
    b = torch.nn.functional.pad(v, (0, -C % block)).unflatten(-1, (-1, block))
    most = b.abs().amax(-1)
    if fmt == "nvfp4":
        g = torch.ones((), device=v.device) if scale is None else scale
        s8 = (most / (6 * g)).clamp(max=448).to(torch.float8_e4m3fn)
        s = s8.float() * g
        r = torch.where(s > 0, (1 / s).clamp(max=FLOAT_MAX), 0.0)
        byte = s8.view(torch.uint8)
        byte = torch.where(most.isfinite(), byte, 0x7F)
    else:
        part, power = torch.frexp(most)  # most = part 2^power, part in [0.5, 1): 6 * 2^s = 0.75 * 2^(s + 3)
        e = torch.where(most > 0, (power - 3 + (part > 0.75).int()).clamp(-127, 126), 0).int()
        r = ((127 - e) << 23).view(torch.float32)  # 2^-e
        byte = torch.where(most.isfinite(), e + 127, 0xFF).to(torch.uint8)
    a = b.abs() * r[..., None]
    q = (a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    q = torch.where(most.isfinite()[..., None], q + 8 * (b < 0).byte(), 0)
    return q.flatten(-2)[..., :C], byte


def _scale_values(byte, fmt):
    if fmt == "nvfp4":
        return byte.view(torch.float8_e4m3fn).float()
    b = byte.int()
    return torch.where(b == 0, 0x00400000, torch.where(b == 255, 0x7FC00000, b << 23)).int().view(torch.float32)  # 2^(b - 127)


def _numbers(q, byte, fmt, scale):
    """Codes and scale bytes to float32 values: (code x block scale) x tensor scale."""
    block, C = 16 if fmt == "nvfp4" else 32, q.shape[-1]
    table = torch.tensor(TABLE + tuple(-t for t in TABLE), device=q.device)
    v = table.index_select(0, q.reshape(-1).int()).view(q.shape)
    s = _scale_values(byte, fmt).repeat_interleave(block, -1)[..., :C]
    return v * s if scale is None else v * s * scale


def _unpack(codes, C):
    return torch.stack((codes & 15, codes >> 4), -1).flatten(-2)[..., :C]


def _plain(state):
    op, E, fmt = state["op"], state["experts"], state["fmt"]
    if op == "permute":
        pos, offsets = _sort(state["ids"], E)
        x = state["x"]
        rows = _put(x[:, None].expand(-1, state["topk"], -1), pos)
        return {"rows": rows, "pos": pos, "offsets": offsets, "dx": _take(state["d_rows"], pos).sum(1).to(x.dtype)}
    if op == "unpermute":
        pos, dy, w = state["pos"], state["dy"], state["weights"]
        r = _take(state["rows"], pos)
        y = (r * w[..., None]).sum(1).to(dy.dtype)
        d_rows = _put((dy.float()[:, None] * w[..., None]).to(dy.dtype), pos)
        return {"y": y, "d_rows": d_rows, "d_weights": (r * dy.float()[:, None]).sum(-1)}
    if op == "quantize":
        v = _numbers(*_quantize(state["x"].float(), fmt, state["scale"]), fmt, state["scale"]).bfloat16()
        return v if state["pos"] is None else _put(v[:, None].expand(-1, state["topk"], -1), state["pos"])
    if op == "swiglu":
        g, u = state["x"].float().chunk(2, -1)
        v = _numbers(*_quantize(g / (1 + torch.exp(-g)) * u, fmt, state["scale"]), fmt, state["scale"]).bfloat16()
        inside = torch.arange(v.shape[0], device=v.device) < state["offsets"][-1]
        return torch.where(inside[:, None], v, 0.0)
    offsets, C = state["offsets"], state["cols"]
    P, N = state["a_codes"].shape[0], state["w_codes"].shape[1]
    i = torch.arange(P, device="cuda")
    e = _expert_of(offsets, i, E)
    j = i - offsets[e].long()
    inside = i < offsets[-1]
    blocks = -(-C // (16 if fmt == "nvfp4" else 32))
    sa = state["a_scales"][offsets[e].long() // 128 + e + j // 128, :, j % 32, j % 128 // 32].flatten(1)[:, :blocks]
    a = _numbers(_unpack(state["a_codes"], C), sa, fmt, None)
    sw = state["w_scales"].permute(0, 1, 4, 3, 2, 5).flatten(4).flatten(1, 3)[:, :N, :blocks]
    w = _numbers(_unpack(state["w_codes"], C), sw, fmt, None)
    at = torch.where(inside, e * state["most"] + j, E * state["most"])  # a row past the last expert is left out
    padded = torch.zeros(E * state["most"] + 1, C, device="cuda").index_copy(0, at, a)
    y = torch.bmm(padded[:-1].view(E, -1, C), w.transpose(1, 2)).view(-1, N)[at.clamp(max=E * state["most"] - 1)]
    if fmt == "nvfp4":
        y = y * (state["a_scale"] * state["w_scale"])[e][:, None]
    return torch.where(inside[:, None], y, 0.0).bfloat16()


def run(state):
    if not own:
        return _plain(state)
    from lora_moe_expert_info_gb300 import fp4, permute
    op, fmt = state["op"], state["fmt"]
    if op == "permute":
        rows, pos, offsets = permute.moe_permute(state["x"], state["ids"], state["experts"], check=False)
        return {"rows": rows, "pos": pos, "offsets": offsets, "dx": permute.moe_permute_backward(state["d_rows"], pos)}
    if op == "unpermute":
        y = permute.moe_unpermute(state["rows"], state["pos"], state["weights"])
        d_rows, d_weights = permute.moe_unpermute_backward(state["dy"], state["rows"], state["pos"], state["weights"])
        return {"y": y, "d_rows": d_rows, "d_weights": d_weights}
    if op == "quantize" and state["pos"] is None:
        codes, scales = fp4.fp4_quantize(state["x"], fmt, state["scale"])
        return fp4.fp4_dequantize(codes, scales, state["cols"], fmt, state["scale"])
    if op == "quantize":
        codes, scales = fp4.fp4_quantize_permuted(state["x"], state["ids"], state["pos"], state["offsets"], fmt, state["scale"])
        return fp4.fp4_dequantize(codes, scales, state["cols"], fmt, state["scale"], expert_offsets=state["offsets"])
    if op == "swiglu":
        codes, scales = fp4.fp4_quantize_swiglu(state["x"], state["offsets"], fmt, state["scale"])
        return fp4.fp4_dequantize(codes, scales, state["cols"], fmt, state["scale"], expert_offsets=state["offsets"])
    return fp4.fp4_expert_product(state["a_codes"], state["a_scales"], state["offsets"], state["w_codes"], state["w_scales"],
                                  state["cols"], fmt, state["a_scale"], state["w_scale"], check=False)


# ------------------------------------------------------------- definition --
def _rounded(v, fmt, g):
    """Float64 values [R, C] after 4-bit quantisation, from the format's definition."""
    block, C = 16 if fmt == "nvfp4" else 32, v.shape[-1]
    b = torch.nn.functional.pad(v, (0, -C % block)).unflatten(-1, (-1, block))
    most = b.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        t = (most / (6 * g)).clamp(max=448)
        step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
        s = torch.round(t / step) * step * g
    else:
        s = torch.exp2(torch.where(most > 0, torch.ceil(torch.log2(most / 6)).clamp(-127, 127), 0.0))
    a = torch.where(s > 0, b.abs() / s, 0.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0)).double()
    a = (torch.round(a / step) * step).clamp(max=6)
    return (torch.sign(b) * a * s).flatten(-2)[..., :C]


def exact(case, seed):
    state = prepare(case, seed)
    op, E, K, fmt = case["op"], case["experts"], case["topk"], case.get("fmt")
    P = _rows(case)
    if K:
        ids = state["ids"].reshape(-1)
        masked = (ids < 0) | (ids >= E)
        # the place of a pair: how many pairs have a smaller id, or the same id and a smaller number
        key = torch.where(masked, E, ids).long() * P + torch.arange(P, device="cuda")
        order = torch.argsort(key)
        token = order // K
        held = ~masked[order]
    if op == "permute":
        dx = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
        rows = torch.where(held[:, None], state["x"][token].double(), 0.0)
        for k in range(K):  # one pair of each token at a time: no two writes meet
            sel = held & (order % K == k)
            dx[token[sel]] += state["d_rows"][sel].double()
        return {"rows": rows, "pos": None, "offsets": None, "dx": dx}
    if op == "unpermute":
        y = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
        w = state["weights"].reshape(-1).double()[order]
        for k in range(K):
            sel = held & (order % K == k)
            y[token[sel]] += state["rows"][sel].double() * w[sel, None]
        dy = state["dy"].double()[token]
        d_w = torch.zeros(P, dtype=torch.float64, device="cuda")
        d_w[order] = torch.where(held, torch.einsum("ph,ph->p", dy, torch.where(held[:, None], state["rows"].double(), 0.0)), 0.0)
        return {"y": y, "d_rows": torch.where(held[:, None], dy * w[:, None], 0.0), "d_weights": d_w.view(-1, K)}
    g = state["scale"].double() if state.get("scale") is not None else 1.0
    if op == "quantize":
        v = _rounded(state["x"].double(), fmt, g)
        return torch.where(held[:, None], v[token], 0.0) if K else v
    if op == "swiglu":
        x = state["x"].double()
        n = case["hidden"]
        h = x[:, :n] * torch.sigmoid(x[:, :n]) * x[:, n:]
        return torch.where(held[:, None], _rounded(h, fmt, g), 0.0)
    C, N = case["hidden"], case["outputs"]
    y = torch.zeros(P, N, dtype=torch.float64, device="cuda")
    first = [int(v) for v in state["offsets"].cpu()]
    values = torch.tensor([(-1) ** (c // 8) * TABLE[c % 8] for c in range(16)], dtype=torch.float64, device="cuda")
    block = 16 if fmt == "nvfp4" else 32

    def matrix(codes, atoms):
        """Codes [R, .] and atoms [row blocks, groups, 32, 4, 4] of one matrix as float64 [R, C]."""
        v = torch.zeros(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device="cuda")
        v[:, 0::2], v[:, 1::2] = values[(codes % 16).long()], values[(codes // 16).long()]
        b = atoms.permute(0, 3, 2, 1, 4).reshape(atoms.shape[0] * 128, -1)[: codes.shape[0]]
        if fmt == "nvfp4":
            m, e = (b % 8).double(), (b // 8).double()
            s = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m * 2.0 ** -9)
        else:
            s = torch.exp2(b.double() - 127)
        return v[:, :C] * s.repeat_interleave(block, 1)[:, :C]

    for e in range(E):
        lo, hi = first[e], first[e + 1]
        if hi > lo:
            at = lo // 128 + e
            a = matrix(state["a_codes"][lo:hi], state["a_scales"][at:at + -(-(hi - lo) // 128)])
            y[lo:hi] = a @ matrix(state["w_codes"][e], state["w_scales"][e]).T
            if fmt == "nvfp4":
                y[lo:hi] *= state["a_scale"].double() * state["w_scale"][e].double()
    return y
