"""Plain restatements of the expert sort and the 4-bit formats, for the tests.

Loops and dense arrays in numpy, in 64 bits except where a format's decision is
defined by single-precision steps (the NVFP4 block scale).  Nothing here is
shared with the library.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------------- sorting --
def sort_pairs(ids: np.ndarray, E: int):
    """(pair_pos [T, K], offsets [E + 1]): pairs by (expert, p), masked ones last as ~row."""
    flat = ids.reshape(-1)
    valid = [p for p in range(flat.size) if 0 <= flat[p] < E]
    order = sorted(valid, key=lambda p: (flat[p], p)) + [p for p in range(flat.size) if not 0 <= flat[p] < E]
    pos = np.zeros(flat.size, dtype=np.int64)
    for row, p in enumerate(order):
        pos[p] = row if 0 <= flat[p] < E else ~row
    counts = np.bincount(flat[valid], minlength=E) if valid else np.zeros(E, dtype=np.int64)
    return pos.reshape(ids.shape).astype(np.int32), np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def permute(x: np.ndarray, pos: np.ndarray) -> np.ndarray:
    T, K = pos.shape
    rows = np.zeros((T * K, x.shape[1]), dtype=x.dtype)
    for t in range(T):
        for k in range(K):
            if pos[t, k] >= 0:
                rows[pos[t, k]] = x[t]
    return rows


def unpermute(rows: np.ndarray, pos: np.ndarray, w: np.ndarray):
    """(y, sum of |w r|) in 64 bits."""
    T, K = pos.shape
    y = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(y)
    for t in range(T):
        for k in range(K):
            if pos[t, k] >= 0:
                y[t] += float(w[t, k]) * rows[pos[t, k]]
                mag[t] += abs(float(w[t, k])) * np.abs(rows[pos[t, k]])
    return y, mag


def unpermute_backward(dy: np.ndarray, rows: np.ndarray, pos: np.ndarray, w: np.ndarray):
    """(d_rows, d_weights, sum of |dy r|) in 64 bits."""
    T, K = pos.shape
    d_rows = np.zeros(rows.shape)
    dw = np.zeros((T, K))
    mag = np.zeros((T, K))
    for t in range(T):
        for k in range(K):
            if pos[t, k] >= 0:
                d_rows[pos[t, k]] = float(w[t, k]) * dy[t]
                dw[t, k] = float(dy[t] @ rows[pos[t, k]])
                mag[t, k] = float(np.abs(dy[t]) @ np.abs(rows[pos[t, k]]))
    return d_rows, dw, mag


# --------------------------------------------------------------- 4-bit floats --
def e4m3_value(b: int) -> float:
    """The value of an unsigned E4M3 byte (0x7f: NaN)."""
    e, m = b >> 3, b & 7
    return float("nan") if b == 0x7F else (m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))


E4M3 = np.array([e4m3_value(b) for b in range(0x7F)])  # increasing


def round_e4m3(v: float) -> int:
    """The byte nearest to 0 <= v <= 448, ties to the even byte."""
    d = np.abs(E4M3 - v)
    best = np.flatnonzero(d == d.min())
    return int(best[0] if best.size == 1 or best[0] % 2 == 0 else best[1])


def round_e2m1(v: float) -> int:
    """The code (0..7) nearest to v >= 0, ties to the even code, saturating."""
    d = np.abs(E2M1 - min(v, 6.0))
    best = np.flatnonzero(d == d.min())
    return int(best[0] if best.size == 1 or best[0] % 2 == 0 else best[1])


def block_scale(most: float, fmt: str, g: float = 1.0):
    """(byte, scale value including g, what a value is multiplied by) of a block
    with largest magnitude `most`; the NVFP4 steps are rounded to float32."""
    f = np.float32
    if not np.isfinite(most):
        return (0xFF if fmt == "mxfp4" else 0x7F), float("nan"), 0.0
    if fmt == "mxfp4":
        s = 0
        if most > 0:
            s = -127
            while most > 6 * 2.0 ** s:
                s += 1
        return s + 127, 2.0 ** s, 2.0 ** -s
    if most == 0:  # whatever g is
        return 0, 0.0, 0.0
    with np.errstate(over="ignore", divide="ignore", under="ignore"):
        t = min(f(most) / (f(6) * f(g)), f(448))
        b = round_e4m3(float(t))
        d = f(f(E4M3[b]) * f(g))
        r = min(f(1) / d, np.finfo(f).max) if d > 0 else f(0)
    return b, float(E4M3[b]) * float(f(g)), float(r)


def quantize_row(x: np.ndarray, fmt: str, g: float = 1.0):
    """(codes 0..15 [C], scale bytes, scale values) of one row of float32 values."""
    n = 16 if fmt == "nvfp4" else 32
    codes = np.zeros(x.size, dtype=np.uint8)
    byts, vals = [], []
    for c in range(0, x.size, n):
        b = x[c:c + n].astype(np.float64)
        most = np.inf if not np.isfinite(b).all() else float(np.abs(b).max())
        byte, val, r = block_scale(most, fmt, g)
        byts.append(byte)
        vals.append(val)
        if np.isfinite(most):
            for i, v in enumerate(b):
                a = float(np.float32(abs(v)) * np.float32(r))
                codes[c + i] = round_e2m1(a) + (8 if np.signbit(v) else 0)
    return codes, np.array(byts, dtype=np.uint8), np.array(vals)


def code_values(codes: np.ndarray) -> np.ndarray:
    return np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]


def unpack_codes(packed: np.ndarray, cols: int) -> np.ndarray:
    """uint8 [rows, pitch] to codes [rows, cols]."""
    out = np.zeros((packed.shape[0], 2 * packed.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out[:, :cols]


def scale_byte_of(scales: np.ndarray, block_row: int, r: int, c: int) -> int:
    """Scale block c of row r of a 128-row block in scales [blocks, atoms, 32, 4, 4]."""
    return int(scales[block_row, c // 4, r % 32, r // 32, c % 4])


def unpack_scales(scales: np.ndarray, place, rows: int, cols: int, fmt: str) -> np.ndarray:
    """Scale values [rows, blocks]; place(row) gives (128-row block, row inside it)."""
    n = -(-cols // (16 if fmt == "nvfp4" else 32))
    out = np.zeros((rows, n))
    for i in range(rows):
        b, r = place(i)
        for c in range(n):
            v = scale_byte_of(scales, b, r, c)
            out[i, c] = e4m3_value(v) if fmt == "nvfp4" else (float("nan") if v == 255 else 2.0 ** (v - 127))
    return out


def numbers(packed: np.ndarray, scales: np.ndarray, place, cols: int, fmt: str) -> np.ndarray:
    """Code x block scale [rows, cols] in 64 bits."""
    n = 16 if fmt == "nvfp4" else 32
    s = unpack_scales(scales, place, packed.shape[0], cols, fmt)
    return code_values(unpack_codes(packed, cols)) * np.repeat(s, n, axis=1)[:, :cols]


def sorted_place(offsets: np.ndarray):
    """place(row) of rows sorted by expert."""
    def place(i):
        e = int(np.searchsorted(offsets, i, side="right")) - 1
        j = i - int(offsets[e])
        return int(offsets[e]) // 128 + e + j // 128, j % 128
    return place
