"""Router loss in NumPy FP64: balance loss over segments, z-loss, per-expert counts, and the gradient to the logits.

A token counts if a segment holds it, its mask entry is not 0 and not all of its logits are -inf. Over the counted
tokens of segment s (n_s of them): L_bal = mean over segments with n_s > 0 of E sum_e (counts / (n_s k)) (probs / n_s),
L_z = mean of lse^2 over every counted token, loss = balance_coef L_bal + z_coef L_z.
"""
from __future__ import annotations

from typing import Dict, Optional

import numpy as np


def _segments(T, seg_offsets):
    off = np.array([0, T]) if seg_offsets is None else np.clip(np.asarray(seg_offsets, dtype=np.int64), 0, T)
    seg = np.full(T, -1, dtype=np.int64)
    for s in range(len(off) - 1):
        seg[off[s]:off[s + 1]] = s
    return seg, len(off) - 1


def router_loss(logits, idx, k: int, balance_coef: float, z_coef: float, seg_offsets=None,
                mask: Optional[np.ndarray] = None) -> Dict[str, np.ndarray]:
    lg = np.asarray(logits, dtype=np.float64)
    T, E = lg.shape
    seg, S = _segments(T, seg_offsets)
    if mask is not None:
        seg = np.where(np.asarray(mask) != 0, seg, -1)
    seg = np.where(np.all(np.isneginf(lg), axis=1), -1, seg)
    live = seg >= 0
    lse, p = np.zeros(T), np.zeros((T, E))
    with np.errstate(invalid="ignore", over="ignore"):
        m = lg[live].max(axis=1, keepdims=True) if live.any() else np.zeros((0, 1))
        ex = np.exp(lg[live] - m)
        lse[live] = (m + np.log(ex.sum(axis=1, keepdims=True)))[:, 0]
        p[live] = ex / ex.sum(axis=1, keepdims=True)
    tokens, counts, probs = np.zeros(S, dtype=np.int64), np.zeros((S, E), dtype=np.int64), np.zeros((S, E))
    bal = 0.0
    for s in range(S):
        rows = np.nonzero(seg == s)[0]
        tokens[s] = len(rows)
        counts[s] = np.bincount(np.asarray(idx)[rows].reshape(-1), minlength=E)
        probs[s] = p[rows].sum(axis=0)
        if len(rows):
            bal += E * np.sum(counts[s] / (len(rows) * k) * probs[s] / len(rows))
    full, n = int(np.count_nonzero(tokens)), int(tokens.sum())
    bal = bal / full if full else 0.0
    z = float(np.sum(lse[live] ** 2)) / n if n else 0.0
    return {"seg": seg, "p": p, "lse": lse, "seg_counts": counts, "seg_probs": probs,
            "seg_tokens": np.concatenate([tokens, [n, full]]), "loss": np.array([balance_coef * bal + z_coef * z, bal, z])}


def router_loss_bwd(f, k: int, balance_coef: float, z_coef: float, dloss: float = 1.0) -> np.ndarray:
    """d(dloss * loss) / dlogits from router_loss's result."""
    p, seg = f["p"], f["seg"]
    S, E = f["seg_counts"].shape
    n, full = int(f["seg_tokens"][S]), int(f["seg_tokens"][S + 1])
    out = np.zeros_like(p)
    for s in range(S):
        rows = np.nonzero(seg == s)[0]
        if not len(rows):
            continue
        w = balance_coef * E * f["seg_counts"][s] / (full * len(rows) ** 2 * k)
        pr = p[rows]
        out[rows] = dloss * pr * (w - (pr @ w)[:, None] + 2.0 * z_coef / n * f["lse"][rows][:, None])
    return out


def grad_bound(f, k: int, balance_coef: float, z_coef: float, dloss: float = 1.0) -> np.ndarray:
    """Magnitude of the terms that router_loss_bwd adds up, with the coefficients centred on a balanced load."""
    p, seg = f["p"], f["seg"]
    S, E = f["seg_counts"].shape
    n, full = int(f["seg_tokens"][S]), int(f["seg_tokens"][S + 1])
    out = np.zeros_like(p)
    for s in range(S):
        rows = np.nonzero(seg == s)[0]
        if not len(rows):
            continue
        w = np.abs(balance_coef * (E * f["seg_counts"][s] / (len(rows) * k) - 1.0) / (full * len(rows)))
        pr = p[rows]
        out[rows] = abs(dloss) * pr * (w + (pr @ w)[:, None] + np.abs(2.0 * z_coef / n * f["lse"][rows])[:, None])
    return out
