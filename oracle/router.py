"""Plain restatements of the norm, the router's choice, the balance loss and their
gradients, for the tests: numpy in 64 bits, the choice in loops.  Roundings to fewer
bits are those that the definitions name.  Nothing here is shared with the library.
"""
from __future__ import annotations

import numpy as np

E4M3 = np.array(sorted({(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)}
                       | {m * 2.0 ** -9 for m in range(8)}))  # by code: 0, 2^-9, ... 448


# ---------------------------------------------------------------------- norm --
def norm(r: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    return r * w / np.sqrt((r * r).mean(1, keepdims=True) + eps)


def norm_backward(dy, r, w, eps, d_r=None):
    """(dx, dw, magnitude of dx's terms, of dw's)."""
    m = 1 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    h = dy * w
    back = r * m * m * (h * r).mean(1, keepdims=True)
    dx = m * (h - back)
    mag = m * (np.abs(h) + np.abs(r) * m * m * np.abs(h * r).mean(1, keepdims=True))
    if d_r is not None:
        dx, mag = dx + d_r, mag + np.abs(d_r)
    return dx, (dy * r * m).sum(0), mag, np.abs(dy * r * m).sum(0)


def eight_bits(y: np.ndarray):
    """(codes uint8 [T, H], exps uint8 [T, groups]) of finite y."""
    T, H = y.shape
    groups = -(-H // 128)
    codes, exps = np.zeros((T, H), np.uint8), np.zeros((T, groups), np.uint8)
    for t in range(T):
        for g in range(groups):
            v = y[t, 128 * g:128 * (g + 1)]
            most = np.abs(v).max()
            s = 0 if most == 0 else max(-127, int(np.ceil(np.log2(most / 448))))
            while s > -127 and most <= 448 * 2.0 ** (s - 1) and most > 0:
                s -= 1
            while most > 448 * 2.0 ** s:
                s += 1
            exps[t, g] = s + 127
            a = np.abs(v) * 2.0 ** -s
            hi = np.clip(np.searchsorted(E4M3, a), 0, len(E4M3) - 1)
            lo = np.maximum(hi - 1, 0)
            near = np.where((E4M3[hi] - a < a - E4M3[lo]) | ((E4M3[hi] - a == a - E4M3[lo]) & (hi % 2 == 0)), hi, lo)
            codes[t, 128 * g:128 * (g + 1)] = near + 128 * np.signbit(v)
    return codes, exps


def from_eight_bits(codes, exps):
    v = E4M3[np.minimum(codes & 127, len(E4M3) - 1)] * np.where(codes & 128, -1.0, 1.0)
    return v * np.exp2(np.repeat(exps.astype(float), 128, axis=1)[:, :codes.shape[1]] - 127)


# -------------------------------------------------------------------- router --
def finite(logits):
    return np.where(np.isfinite(logits), logits, -np.inf)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-v))


def scores(logits, scoring):
    """softmax or sigmoid [T, E], zeros where a logit is not finite."""
    v = finite(logits)
    if scoring == "sigmoid":
        return np.where(np.isfinite(v), sigmoid(v), 0.0)
    with np.errstate(invalid="ignore"):
        e = np.where(np.isfinite(v), np.exp(v - v.max(1, keepdims=True)), 0.0)
    total = e.sum(1, keepdims=True)
    return e / np.where(total > 0, total, 1)


def choose(logits, K, scoring, bias=None, groups=1, best=1, mask=None):
    T, E = logits.shape
    ids = np.full((T, K), -1, np.int32)
    v = finite(logits)
    key = v.copy()
    if scoring == "sigmoid" and (bias is not None or groups > 1):
        key = np.where(np.isfinite(v), sigmoid(v) + (0 if bias is None else bias), -np.inf)
        key = np.where(np.isfinite(key), key, -np.inf)
    size = E // groups
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        k = key[t].copy()
        if groups > 1:
            value = []
            for g in range(groups):
                top = sorted((x for x in k[g * size:(g + 1) * size] if x > -np.inf), reverse=True)
                value.append(-np.inf if not top else top[0] if scoring == "softmax" else sum(top[:2]))
            order = sorted(range(groups), key=lambda g: (-value[g], g))
            for g in order[best:]:
                k[g * size:(g + 1) * size] = -np.inf
        order = sorted((e for e in range(E) if k[e] > -np.inf), key=lambda e: (-k[e], e))[:K]
        ids[t, :len(order)] = order
    return ids


def taken(ids, E, logits):
    """How often each token's places hold each expert that can be chosen, [T, K, E]."""
    hot = (ids[:, :, None] == np.arange(E)) & np.isfinite(logits)[:, None, :]
    return hot.astype(float)


def weights(logits, ids, scoring, renormalize, scale):
    s = (taken(ids, logits.shape[1], logits) * scores(logits, scoring)[:, None, :]).sum(2)
    if renormalize:
        total = s.sum(1, keepdims=True)
        s = s / np.where(total > 0, total, 1)
    return scale * s


def weights_backward(g, logits, ids, scoring, renormalize, scale):
    """The gradient of sum(g weights) by the logits, from the Jacobians of each step."""
    E = logits.shape[1]
    hot, s = taken(ids, E, logits), scores(logits, scoring)
    u = (hot * s[:, None, :]).sum(2)
    g = scale * g
    if renormalize:
        total = u.sum(1, keepdims=True)
        safe = np.where(total > 0, total, 1)
        g = np.where(total > 0, (g - (g * u).sum(1, keepdims=True) / safe) / safe, 0)
    gs = (hot * g[:, :, None]).sum(1)
    if scoring == "sigmoid":
        return gs * s * (1 - s)
    return s * (gs - (gs * s).sum(1, keepdims=True))


def balance(logits, ids, scoring, mask=None):
    """(loss, counts [E + 1])."""
    T, E = logits.shape
    K = ids.shape[1]
    keep = np.ones(T, bool) if mask is None else mask
    n = int(keep.sum())
    counts = np.array([((ids == e) & keep[:, None]).sum() for e in range(E)] + [n])
    s = scores(logits, scoring)
    total = s.sum(1, keepdims=True)
    p = np.where(keep[:, None], s / np.where(total > 0, total, 1), 0)
    return float((p.sum(0) * counts[:E]).sum() * E / (K * max(n, 1) ** 2)), counts.astype(np.int32)


def balance_backward(d_loss, logits, counts, K, scoring, mask=None):
    T, E = logits.shape
    a = d_loss * counts[:E] * E / (K * max(int(counts[E]), 1) ** 2)
    s = scores(logits, scoring)
    total = s.sum(1, keepdims=True)
    p = s / np.where(total > 0, total, 1)
    d = p * (a - (p * a).sum(1, keepdims=True)) * (1 if scoring == "softmax" else 1 - s)
    return d if mask is None else np.where(mask[:, None], d, 0)
