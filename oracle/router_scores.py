"""Routing by scores in NumPy FP64: softmax or sigmoid scores, a bias and groups of experts in the choice, gates from the
chosen scores, their gradient to the logits, and the bias update.

The choice is made on c = FP32(s + b), rounded once, and on group scores rounded once to FP32: that rounding decides
integers, so it is followed exactly. NaN logits and sums count as -inf, +inf logits as the largest finite FP32 value.
"""
from __future__ import annotations

import numpy as np

BIG = float(np.finfo(np.float32).max)


def clean(logits):
    lg = np.asarray(logits, dtype=np.float64)
    return np.minimum(np.where(np.isnan(lg), -np.inf, lg), BIG)


def scores(logits, score: str):
    """s [T, E] in FP64; a softmax row without a logit above -inf is 0 everywhere."""
    lg = clean(logits)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-lg))
        m = lg.max(axis=1, keepdims=True)
        ex = np.where(np.isneginf(m), 0.0, np.exp(lg - m))
        den = ex.sum(axis=1, keepdims=True)
        return np.where(den > 0, ex / np.where(den > 0, den, 1.0), 0.0)


def _f32(x):
    with np.errstate(over="ignore", invalid="ignore"):
        x = np.asarray(x, dtype=np.float64).astype(np.float32)
    return np.where(np.isnan(x), np.float32(-np.inf), x).astype(np.float64)


def choose(s, bias, k: int, n_groups=1, topk_groups=1, group_top=1):
    """idx [T, k]: the k largest c of the eligible groups, largest first, ties to the lower index."""
    T, E = s.shape
    with np.errstate(invalid="ignore"):
        c = _f32(s if bias is None else s + np.asarray(bias, dtype=np.float64))
    size = E // n_groups
    open_ = np.ones((T, E), dtype=bool)
    if n_groups > 1:
        per = -np.sort(-c.reshape(T, n_groups, size), axis=2)[:, :, :min(group_top, size)]
        with np.errstate(invalid="ignore"):
            rank = _f32(per.sum(axis=2))
        best = np.argsort(-rank, axis=1, kind="stable")[:, :topk_groups]
        g = np.zeros((T, n_groups), dtype=bool)
        np.put_along_axis(g, best, True, axis=1)
        open_ = np.repeat(g, size, axis=1)
    # eligible experts in front of the others, then by c, then by index
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -c, ~open_), axis=1)
    return order[:, :k].astype(np.int32)


def gates(logits, idx, score: str, renormalize: bool, scale: float):
    s = np.take_along_axis(scores(logits, score), idx.astype(np.int64), axis=1)
    if renormalize:
        # relative to the largest chosen logit: scores far below the range of FP64 keep their ratio
        z = np.take_along_axis(clean(logits), idx.astype(np.int64), axis=1)
        low = z if score == "softmax" else np.minimum(z, 0.0)
        top = low.max(axis=1, keepdims=True)
        with np.errstate(invalid="ignore"):
            u = np.where(np.isneginf(top), 0.0, np.exp(low - top))
        if score == "sigmoid":
            u = u / (1.0 + np.exp(-np.abs(z)))
        den = u.sum(axis=1, keepdims=True)
        s = np.where(den > 0, u / np.where(den > 0, den, 1.0), 0.0)
    return scale * s


def route(logits, bias, k, score, n_groups=1, topk_groups=1, group_top=1, renormalize=True, scale=1.0):
    idx = choose(scores(logits, score), bias, k, n_groups, topk_groups, group_top)
    return idx, gates(logits, idx, score, renormalize, scale)


def backward(logits, idx, dgates, score, renormalize=True, scale=1.0):
    """dlogits [T, E] of gates(): the chosen experts are constant."""
    lg, ix = clean(logits), idx.astype(np.int64)
    dg = np.asarray(dgates, dtype=np.float64)
    out = np.zeros(lg.shape)
    z = np.take_along_axis(lg, ix, axis=1)
    with np.errstate(over="ignore"):
        rest = 1.0 / (1.0 + np.exp(z)) if score == "sigmoid" else 1.0
    if renormalize:
        gh = gates(logits, idx, score, True, 1.0)
        np.put_along_axis(out, ix, scale * gh * rest * (dg - (gh * dg).sum(axis=1, keepdims=True)), axis=1)
        return out
    s = scores(logits, score)
    sel = np.take_along_axis(s, ix, axis=1)
    if score == "sigmoid":
        np.put_along_axis(out, ix, scale * sel * rest * dg, axis=1)
        return out
    np.put_along_axis(out, ix, dg, axis=1)
    return scale * s * (out - (sel * dg).sum(axis=1, keepdims=True))


def backward_bound(logits, idx, dgates, score, renormalize=True, scale=1.0):
    """Magnitude of the terms that backward() adds up."""
    ix = idx.astype(np.int64)
    dg = np.abs(np.asarray(dgates, dtype=np.float64))
    out = np.zeros(np.asarray(logits).shape)
    z = np.take_along_axis(clean(logits), ix, axis=1)
    with np.errstate(over="ignore"):
        rest = 1.0 / (1.0 + np.exp(z)) if score == "sigmoid" else 1.0
    if renormalize:
        gh = gates(logits, idx, score, True, 1.0)
        np.put_along_axis(out, ix, abs(scale) * gh * rest * (dg + (gh * dg).sum(axis=1, keepdims=True)), axis=1)
        return out
    s = scores(logits, score)
    sel = np.take_along_axis(s, ix, axis=1)
    if score == "sigmoid":
        np.put_along_axis(out, ix, abs(scale) * sel * rest * dg, axis=1)
        return out
    np.put_along_axis(out, ix, dg, axis=1)
    return abs(scale) * s * (out + (sel * dg).sum(axis=1, keepdims=True))


def bias_update(bias, counts, rate):
    """FP32 bias after one step: up where an expert has less than the mean load, down where it has more."""
    load = np.asarray(counts, dtype=np.int64).sum(axis=0)
    sign = np.sign(load.sum() - load.size * load).astype(np.float32)
    return np.asarray(bias, dtype=np.float32) + sign * np.float32(rate)
