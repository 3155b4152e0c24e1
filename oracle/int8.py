"""8-bit integer expert path in NumPy: symmetric per-row quantisation with the kernel's FP32 steps (an integer is
decided by floating point there), exact integer products, and the forward in FP64 around them.
"""
from __future__ import annotations

import numpy as np

from .ffn import combine, silu
from .routing import dispatch, layout, route


def quantize_rows(a: np.ndarray):
    """Codes (int8) and scale (FP32) of every row of [..., cols]: amax / 127 and RNE(v * (127 / amax)), each step one
    FP32 rounding. A row of zeros, or of values whose multiplier overflows, has codes 0 and scale 1; a row that is not
    finite has codes 0 and scale NaN."""
    a = np.asarray(a, dtype=np.float32)
    bad = ~np.all(np.isfinite(a), axis=-1, keepdims=True)
    amax = np.max(np.where(bad, np.float32(0), np.abs(a)), axis=-1, keepdims=True) if a.shape[-1] else np.zeros(
        a.shape[:-1] + (1,), np.float32)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        inv = np.float32(127) / amax
        ok = (amax > 0) & np.isfinite(inv)
        q = np.clip(np.rint(np.where(ok & ~bad, a, np.float32(0)) * np.where(ok, inv, np.float32(0))), -127, 127)
        scale = np.where(bad, np.float32(np.nan), np.where(ok, amax / np.float32(127), np.float32(1)))
    return q.astype(np.int8), scale[..., 0].astype(np.float32)


def matmul(xq, xs, wq, ws, offsets=None):
    """y [rows, N] in FP64: exact integer products of the rows of each group with its weights, times both scales. Rows
    in no group are NaN."""
    rows, G, N = xq.shape[0], wq.shape[0], wq.shape[1]
    off = np.array([0, rows]) if offsets is None else np.clip(np.asarray(offsets, dtype=np.int64), 0, rows)
    y = np.full((rows, N), np.nan)
    for g in range(G):
        a, b = off[g], max(off[g], off[g + 1])
        acc = xq[a:b].astype(np.float64) @ wq[g].astype(np.float64).T  # |sum| < 2^31: exact in FP64
        y[a:b] = acc * xs[a:b, None].astype(np.float64) * ws[g][None].astype(np.float64)
    return y


def decode_yd(codes):
    """Values of the 16-bit rows between the experts and combine: sign, 7 exponent bits (bias 63), 8 mantissa bits,
    subnormal below 2^-62; 0x7fff is NaN."""
    c = codes.astype(np.int64) & 0xffff
    e, m = (c >> 8) & 0x7f, c & 0xff
    v = np.where(e > 0, np.ldexp(1.0 + m / 256.0, e - 63), np.ldexp(m / 256.0, -62))
    v = np.where(c >> 15, -v, v)
    return np.where((c & 0x7fff) == 0x7fff, np.nan, v)


def forward(x, logits, w1q, w1s, w2q, w2s, *, k, e0, E_local, n_chunks, P_c):
    """Layer forward on integer codes. Returns the routing state and h, yd, out in FP64 (h quantised from its FP32
    rounding, the value that the kernel holds)."""
    idx, gates = route(logits, k)
    E = logits.shape[1]
    counts, offsets, row_of, src_token = layout(idx, E, e0, E_local, n_chunks, P_c)
    xq, xs = quantize_rows(x)
    xdq = dispatch(xq.astype(np.int64), src_token).astype(np.int8)
    xds = np.ones(src_token.size, dtype=np.float32)
    v = src_token >= 0
    xds[v] = xs[src_token[v]]
    I, P, H = w1q.shape[1] // 2, src_token.size, x.shape[1]
    h, yd = np.zeros((P, I)), np.zeros((P, H))
    for c in range(n_chunks):
        for e in range(E_local):
            r0, r1 = c * P_c + int(offsets[c, e]), c * P_c + int(offsets[c, e + 1])
            if r1 == r0:
                continue
            gu = matmul(xdq[r0:r1], xds[r0:r1], w1q[e:e + 1], w1s[e:e + 1])
            h[r0:r1] = silu(gu[:, :I]) * gu[:, I:]
            hq, hs = quantize_rows(h[r0:r1].astype(np.float32))
            yd[r0:r1] = matmul(hq, hs, w2q[e:e + 1], w2s[e:e + 1])
    return dict(idx=idx, gates=gates, counts=counts, offsets=offsets, row_of=row_of, src_token=src_token, xdq=xdq,
                xds=xds, h=h, yd=yd, out=combine(yd, gates, row_of))
