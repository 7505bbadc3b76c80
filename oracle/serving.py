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

__all__ = ["attention", "heads", "adapters", "tables", "sample"]

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


def tables(change, lens, table, page, tokens, ring=None, free=(0, 0), offsets=None):
    """One step of lutgemm_batch_tables, sequence by sequence, in whole numbers. table and ring
    are lists that are updated; returns (positions, slots, lens, starts, free)."""
    seqs, width = len(change), len(table[0]) if table else 0
    limit = width * page
    first, count = (free[0] % len(ring), min(max(free[1], 0), len(ring))) if ring else (0, 0)
    positions, slots, after, starts = [], [], [], [0]
    taken, given, stop = 0, [], False
    old = list(ring) if ring else []
    for s in range(seqs):
        n, d = min(max(lens[s], 0), limit), change[s]
        held = -(-n // page)
        if d < 0:
            left = max(0, n + d)
            if ring:
                given += table[s][-(-left // page):held]
            n = left
        elif 0 < d <= limit - n:
            more = -(-(n + d) // page) - held if ring else 0
            stop = stop or len(positions) + d > tokens or taken + more > count
            if not stop:
                for j in range(more):
                    table[s][held + j] = old[(first + taken + j) % len(old)]
                taken += more
                for i in range(n, n + d):
                    positions.append(i + (offsets[s] if offsets else 0))
                    slots.append(table[s][i // page] * page + i % page)
                n += d
        after.append(n)
        starts.append(len(positions))
    rest = tokens - len(positions)
    positions, slots = positions + [0] * rest, slots + [-1] * rest
    if not ring:
        return positions, slots, after, starts, None
    given = given[:len(ring) - count]
    for j, x in enumerate(given):
        ring[(first + count + j) % len(ring)] = x
    return positions, slots, after, starts, [(first + taken) % len(ring), count - taken + len(given)]


def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row of lutgemm_sample_tokens: (token, log-probability, margin): how far, of the
    total, the nearest border of the token and of the filters is from moving."""
    x = np.asarray(x, np.float64)
    if (not (x < np.inf).all() or not (x > -np.inf).any() or not 0 <= u < 1
            or not 0 <= temperature < np.inf or top_p != top_p or min_p != min_p):
        return -1, np.nan, 1.0
    if temperature == 0:
        return int(np.argmax(x)), 0.0, 1.0
    order = np.argsort(-x, kind="stable")
    with np.errstate(over="ignore"):
        w = np.exp((x[order] - x[order[0]]) / temperature)
    margin = 1.0
    if top_k > 0:
        w[top_k:] = 0
    if top_p < 1:
        upto, total = np.cumsum(w), w.sum()
        end = min(int(np.searchsorted(upto, top_p * total)), len(w) - 1)
        if w[:end + 1].min() != w[:end + 1].max():  # sums of equal weights are exact
            margin = min(abs(upto[end] - top_p * total), abs(upto[end] - w[end] - top_p * total)) / total
        w[max(1, end + 1):] = 0
    if min_p > 0:
        least = min(min_p, 1.0)
        near = np.abs(w[w > 0] - least)
        near = near[near > 0]
        margin = min(margin, near.min() if near.size else 1.0)
        w[w < least] = 0
    kept = np.zeros_like(w)
    kept[order] = w
    upto = np.cumsum(kept)
    goal = u * upto[-1]
    i = int(np.searchsorted(upto, goal, side="right"))
    if w.max() != w[w > 0].min():
        below = upto[i] - kept[i]
        margin = min(margin, (upto[i] - goal) / upto[-1], (goal - below) / upto[-1] if u > 0 else 1.0)
    return i, float(np.log(kept[i]) - np.log(upto[-1])), float(margin)
