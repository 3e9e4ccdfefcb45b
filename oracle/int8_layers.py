"""Definitions in 64 bits of the operators with 8-bit weights (include/dq4_int8.h): TEST
INFRASTRUCTURE ONLY, like the rest of this package.

Arrays are numpy; 16-bit activations come as float64 arrays of their values.  A weight is codes
CB [N, K] and scales SCB [N]: values CB * SCB / 127.
"""

from __future__ import annotations

import numpy as np

TINY = 2.0 ** -100
R127 = np.float32(1.0) / np.float32(127.0)


def quantize(x, threshold=0.0, max_outliers=64):
    """(codes, scales, cols, outliers, count) of rows x; the last three None without a
    threshold."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    loud = np.abs(x) >= threshold if threshold else np.zeros(x.shape, bool)
    codes = np.zeros((M, K), np.int8)
    scales = np.zeros(M)
    for m in range(M):
        rest = np.abs(x[m][~loud[m]])
        top = rest.max() if rest.size else 0.0
        if np.isnan(rest).any() or top == np.inf:
            scales[m] = np.nan
            continue
        if top < TINY:
            continue
        scales[m] = top
        inverse = np.float32(127.0) / np.float32(top)
        with np.errstate(invalid="ignore", over="ignore"):
            v = np.rint((x[m].astype(np.float32) * inverse).astype(np.float64))
        codes[m] = np.clip(v, -127, 127).astype(np.int8)
    if not threshold:
        return codes, scales, None, None, None
    found = np.flatnonzero(loud.any(0))
    kept = found[:max_outliers]
    codes[:, kept] = 0
    cols = np.full(max_outliers, -1, np.int64)
    cols[:len(kept)] = kept
    outliers = np.zeros((M, max_outliers))
    outliers[:, :len(kept)] = x[:, kept]
    return codes, scales, cols, outliers, len(found)


def used_columns(cols, K):
    """(entry, column) of the columns that count: in range and above all before them."""
    top, used = -1, []
    for at, c in enumerate(np.asarray(cols).tolist()):
        if top < c < K:
            top = c
            used.append((at, c))
    return used


def linear(codes, scales, CB, SCB, cols=None, outliers=None, bias=None):
    """(Y, size): the product, and the sum of its terms' magnitudes."""
    a = codes.astype(np.float64) * (np.asarray(scales, np.float64)[:, None] / 127)
    if cols is not None:
        for at, c in used_columns(cols, codes.shape[1]):
            a[:, c] = outliers[:, at]
    w = CB.astype(np.float64) * (np.asarray(SCB, np.float64)[:, None] / 127)
    with np.errstate(invalid="ignore"):
        y, size = a @ w.T, np.abs(a) @ np.abs(w).T
        dead = ~np.isfinite(np.asarray(scales, np.float64))
        if cols is not None:
            for at, _ in used_columns(cols, codes.shape[1]):
                dead |= ~np.isfinite(outliers[:, at])
    if bias is not None:
        y, size = y + bias, size + np.abs(bias)
    y[dead] = np.nan
    return y, size


def weight16(CB, SCB, to16):
    """The weight's values rounded to 16 bits by to16 (float32 -> float32)."""
    w = (CB.astype(np.float32) * np.asarray(SCB, np.float32)[:, None]) * R127
    return to16(w).astype(np.float64)


def linear_backward(dy, w):
    """(dX, size) of dy and the weight's 16-bit values."""
    with np.errstate(invalid="ignore"):
        return dy @ w, np.abs(dy) @ np.abs(w)


def route(logits, top_k, renormalize):
    """(ids, weights) of each token."""
    ids, weights = [], []
    for row in np.asarray(logits, np.float64):
        key = np.where(np.isnan(row), -np.inf, row)
        order = sorted(range(len(row)), key=lambda e: (-key[e], e))[:top_k]
        ids.append(order)
        if np.isnan(row).any():
            weights.append(np.full(top_k, np.nan))
        elif key.max() == -np.inf:
            weights.append(np.zeros(top_k))
        else:
            with np.errstate(invalid="ignore"):
                p = np.exp(row - row.max())
            weights.append(p[order] / (p[order].sum() if renormalize else p.sum()))
    return np.array(ids, np.int32), np.array(weights)


def moe(x, logits, w1, s1, w2, s2, top_k, renormalize):
    """(Y, ids, weights, size, unit): the layer; the sum of the magnitudes of Y's terms, and what
    a relative change of every inner value can move."""
    x = np.asarray(x, np.float64)
    ids, weights = route(logits, top_k, renormalize)
    inner = w2.shape[2]
    y, size, unit = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    for t in range(len(x)):
        for e, p in zip(ids[t], weights[t]):
            if p == 0:
                continue
            w = w1[e].astype(np.float64) * (np.asarray(s1[e], np.float64)[:, None] / 127)
            with np.errstate(invalid="ignore", over="ignore"):
                both, reach = w @ x[t], np.abs(w) @ np.abs(x[t])
                gate, up = both[:inner], both[inner:]
                act = gate / (1 + np.exp(-gate))
                h = act * up
                # silu's slope is below 1.1
                slack = 1.1 * reach[:inner] * np.abs(up) + np.abs(act) * reach[inner:]
                v = w2[e].astype(np.float64) * (np.asarray(s2[e], np.float64)[:, None] / 127)
                y[t] += p * (v @ h)
                size[t] += abs(p) * (np.abs(v) @ np.abs(h))
                unit[t] += abs(p) * (np.abs(v) @ slack)
    return y, ids, weights, size, unit
