"""AdamW in NumPy: the step in FP64, and the 8-bit averages with the FP32 steps that decide their codes.

m = s c|c| / 127^2 (int8 c), v = s (c / 255)^4 (uint8 c), s the largest magnitude of a block of 256 elements. A value
between two codes takes the upper one where (a - below) / (above - below) > r, r from a hash of the element's place,
the step and the seed (1/2 for the nearest code).
"""
from __future__ import annotations

import numpy as np

F = np.float32
BLOCK = 256


def _u32(x):
    return np.asarray(x).astype(np.uint64) & np.uint64(0xffffffff)


def random_bits(places, seed: int, step: int):
    """32 bits per place (the low half rounds m, the high half v) and 16 more (a BF16 weight)."""
    key = ((step & 0xffffffff) * 0x243F6A89 + seed) & 0xffffffff
    key ^= key >> 16
    key = (key * 0xB7E15163) & 0xffffffff
    key ^= key >> 15
    x = _u32(_u32(places) * np.uint64(0x9E3779B9) + np.uint64(key))
    x = _u32((x ^ (x >> np.uint64(16))) * np.uint64(0xB7E15163))
    x = x ^ (x >> np.uint64(15))
    return x, _u32(x * np.uint64(0x243F6A89)) >> np.uint64(16)


def places(sizes):
    """Place of every element: tensors one behind the other, each from a multiple of 256 on."""
    out, at = [], 0
    for n in sizes:
        out.append(np.arange(at, at + n, dtype=np.int64))
        at += -(-n // BLOCK) * BLOCK
    return out


def levels(which: str):
    top = 127 if which == "m" else 255
    t = np.arange(top + 1).astype(F) * F(1.0 / top)
    t = t * t
    return t if which == "m" else t * t


def _blocks(x):
    n = x.size
    full = np.zeros(-(-n // BLOCK) * BLOCK, dtype=F)
    full[:n] = x
    return full.reshape(-1, BLOCK)


def encode(x, which: str, r=None):
    """Codes and scales of FP32 x [n]; r [n]: 16 random bits each (None: nearest)."""
    x = np.asarray(x, dtype=F)
    n = x.size
    per = np.abs(_blocks(x))
    s = per.max(axis=1)
    s = np.where(s < F(2.0 ** -120), F(0), np.where(np.isinf(s), F(np.nan), s)).astype(F)
    inv = np.where(s > 0, F(1) / np.where(s > 0, s, F(1)), F(0)).astype(F)
    a = np.minimum(per * inv[:, None], F(1)).reshape(-1)[:n]
    lev = levels(which)
    c = np.clip(np.searchsorted(lev, a, side="right") - 1, 0, len(lev) - 2)
    lo, hi = lev[c], lev[c + 1]
    frac = F(0.5) if r is None else np.asarray(r).astype(F) * F(2.0 ** -16)
    c = c + (a - lo > frac * (hi - lo))
    if which == "v":
        return np.where(a > 0, np.maximum(c, 1), 0).astype(np.uint8), s
    return np.where(x < 0, -c, c).astype(np.int8), s


def decode(codes, s, which: str):
    """FP32 values of codes [n] with scales [ceil(n / 256)]."""
    n = codes.size
    c = codes.astype(np.int64)
    v = levels(which)[np.abs(c)] * np.repeat(np.asarray(s, dtype=F), BLOCK)[:n]
    return np.where(c < 0, -v, v).astype(F)


def averages(g, m, v, beta1, beta2, grad_scale=1.0):
    """m', v' in FP32, each operation rounded once; g, m, v FP32 values."""
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        x = np.asarray(g, dtype=F) * F(grad_scale)
        return (np.asarray(m, dtype=F) * F(beta1) + x * F(1.0 - beta1),
                np.asarray(v, dtype=F) * F(beta2) + (x * x) * F(1.0 - beta2))


def step(w, g, m, v, lr, beta1, beta2, eps, t, weight_decay=0.0, grad_scale=1.0):
    """w', m', v' in FP64."""
    w, g, m, v = (np.asarray(a, dtype=np.float64) for a in (w, g, m, v))
    x = g * grad_scale
    m = beta1 * m + (1.0 - beta1) * x
    v = beta2 * v + (1.0 - beta2) * x * x
    mh, vh = m / (1.0 - beta1 ** t), v / (1.0 - beta2 ** t)
    return w - lr * weight_decay * w - lr * mh / (np.sqrt(vh) + eps), m, v
