"""Plain fp64 forms of the operators beside the weight products, on the CPU, with
the error bounds that their tests use.

Written from the formulas, row by row, without the library. Each function returns
``(result, bound)``: the exact result of the given (already rounded) inputs and
how far an output computed in fp32 and rounded to the element type may lie from it.
``u`` is half the type's epsilon, the largest relative error of one rounding; fp32
sums of n terms are off by at most n 2^-24 of the sum of the terms' magnitudes.
"""
from __future__ import annotations

import numpy as np

__all__ = ["attention", "heads", "adapters"]

_F32 = 2.0 ** -24


def attention(q, k, v, len_new, n, scale, window, u):
    """One sequence: q [len][H][D], k and v [n][Hk][D] (fp64 arrays). The bound counts
    the rounding of the output (u |o|), of the softmax weights (u A and, where fp16
    weights lose digits, 2^-32 per key against a sum of weights of at least 1: half of its
    smallest number, the largest weight being kept as 2^7 or more), the fp32 sums over the keys, and the error of a score, which moves a
    weight by as much: D products in fp32, the scaling and the base-2 exponential."""
    H, D = q.shape[1:]
    group = H // k.shape[1] if k.shape[1] else 1
    out = np.zeros_like(q)
    tol = np.zeros_like(q)
    for t in range(len_new):
        p = n - len_new + t
        lo = max(0, p - window + 1) if window else 0
        if p < 0 or p + 1 <= lo:
            continue
        for h in range(H):
            kk, vv = k[lo:p + 1, h // group], v[lo:p + 1, h // group]
            s = kk @ q[t, h] * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[t, h] = w @ vv
            size = w @ np.abs(vv)
            ds = (D + 16) * _F32 * scale * (np.abs(kk) @ np.abs(q[t, h])).max() + 2.0 ** -20
            keys = p + 1 - lo
            tol[t, h] = (u * np.abs(out[t, h]) + u * size + 2.0 ** -32 * np.abs(vv).sum(0)
                         + (2 * keys * _F32 + 2 * ds) * (size + np.abs(out[t, h])) + 2.0 ** -25)
    return out, 1.01 * tol


def heads(x, weight, eps, cos, sin, interleaved, u):
    """x [tokens][H][D] fp64, weight [D] or None, cos and sin [tokens][R/2]. The bound
    counts the output's rounding and, in fp32, the sum of D squares, the root, the
    weights and the two products of a pair."""
    D = x.shape[2]
    R = 2 * cos.shape[1]
    x = x.copy()
    if weight is not None:
        x = x / np.sqrt((x ** 2).mean(2, keepdims=True) + eps) * weight
    out, size = x.copy(), np.abs(x)
    i = np.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
    c, s = cos[:, None], sin[:, None]
    out[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
    out[:, :, b] = x[:, :, b] * c + x[:, :, a] * s
    both = np.abs(x[:, :, a]) + np.abs(x[:, :, b])
    size[:, :, a] = both
    size[:, :, b] = both
    return out, u * np.abs(out) + (D + 32) * _F32 * size + 2.0 ** -25


def adapters(y, x, a, b, ids, scales, u, pair):
    """y [m][N], x [m][K], a [L][r][K], b [L][N][r]. The bound counts the output's
    rounding, the fp32 sums of both products, and the rounding of the inner vector to a
    pair of numbers: `pair` of its largest entry."""
    out = y.copy()
    tol = np.zeros_like(y)
    for i, l in enumerate(ids):
        if 0 <= l < a.shape[0]:
            s = 1.0 if scales is None else scales[l]
            t = a[l] @ x[i]
            dt = (x.shape[1] + 64) * _F32 * (np.abs(a[l]) @ np.abs(x[i])) + pair * np.abs(t).max()
            B = np.abs(b[l])
            out[i] += s * (b[l] @ t)
            tol[i] = abs(s) * (B @ dt + (2 * b.shape[2] + 8) * _F32 * (B @ np.abs(t)))
    return out, 1.01 * (u * np.abs(out) + tol + 4 * _F32 * (np.abs(y) + np.abs(out))) + 2.0 ** -25
