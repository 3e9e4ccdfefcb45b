"""64-bit definitions of the attention-side operators, in plain numpy (test infrastructure).

Written from the formulas in include/dq4_attn.h, one head or row at a time; they share no code
with the CUDA path.  The rotation of the cache's append is defined in FP32 with every product
and sum rounded on its own, so there it is computed in float32.
"""

from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
MIN_SCALE = 2.0 ** -100


def rotation_pairs(rotary: int, interleaved: bool):
    """The indices (first, second) of the rotated pairs; pair j turns by table column j."""
    j = np.arange(rotary // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rotary // 2)


def rotate(x: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [..., dim] turned by cos, sin [..., rotary / 2], in x's type."""
    a, b = rotation_pairs(2 * cos.shape[-1], interleaved)
    y = x.copy()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def norm_rope(x, weight, cos, sin, positions, eps, interleaved):
    """(y, magnitude): y in float64, and for each value the sum of the magnitudes of its pair."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    if cos is None:
        return x, np.abs(x)
    c, s = (t.astype(np.float64)[positions][:, None] for t in (cos, sin))
    size = rotate(np.abs(x), np.abs(c), -np.abs(s), interleaved)
    a, b = rotation_pairs(2 * cos.shape[1], interleaved)
    size[..., b] = size[..., a] = np.abs(x[..., a]) + np.abs(x[..., b])
    return rotate(x, c, s, interleaved), size


def norm_rope_backward(dy, x, weight, cos, sin, positions, eps, interleaved):
    """(dx, dx magnitude, dw, dw magnitude) in float64."""
    g = dy.astype(np.float64)
    size = np.abs(g)
    if cos is not None:
        c, s = (t.astype(np.float64)[positions][:, None] for t in (cos, sin))
        a, b = rotation_pairs(2 * cos.shape[1], interleaved)
        size[..., b] = size[..., a] = np.abs(g[..., a]) + np.abs(g[..., b])
        g = rotate(g, c, -s, interleaved)
    if weight is None:
        return g, size, None, None
    x, w = x.astype(np.float64), weight.astype(np.float64)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    dx = r * (g * w - xh * (g * w * xh).mean(-1, keepdims=True))
    dx_size = r * (size * np.abs(w) + np.abs(xh) * (size * np.abs(w * xh)).mean(-1, keepdims=True))
    return dx, dx_size, (g * xh).sum((0, 1)), (size * np.abs(xh)).sum((0, 1))


def e4m3(x: np.ndarray) -> np.ndarray:
    """Round to the nearest e4m3 value, ties to even (|x| <= 448); NaN stays NaN."""
    x = np.asarray(x, np.float64)
    _, power = np.frexp(np.where(np.isfinite(x), x, 1.0))
    step = np.ldexp(1.0, np.maximum(power - 4, -9))
    return np.rint(x / step) * step


def fitting_scale(amax: float) -> float:
    """The least power of two with amax <= 448 * scale, at least 2^-100; NaN if not finite."""
    if not np.isfinite(amax):
        return np.nan
    scale = MIN_SCALE
    while amax > E4M3_MAX * scale:
        scale *= 2
    return scale


def append(codes, scales, x, cos, sin, table, lens, cu, interleaved):
    """Append x [tokens, heads, dim] (float32) to codes [pages, heads, page, dim] (values) and
    scales [pages, heads], in place; cos is None for values."""
    page = codes.shape[2]
    for b, length in enumerate(lens):
        new = x[cu[b]:cu[b + 1]]
        start = length - len(new)
        if cos is not None and len(new):
            pos = np.arange(start, length)
            new = rotate(new, cos[pos][:, None], sin[pos][:, None], interleaved)
        for j in range(start // page, -(-length // page)) if len(new) else ():
            lo, hi = max(start, j * page), min(length, (j + 1) * page)
            for h in range(x.shape[1]):
                part = new[lo - start:hi - start, h].astype(np.float64)
                at = table[b][j], h
                with np.errstate(invalid="ignore"):
                    fit = fitting_scale(np.max(np.abs(part)))
                    old = float(scales[at]) if lo > j * page else 0.0
                    scale = np.nan if np.isnan(fit) or np.isnan(old) else max(old, fit)
                    first = lo - j * page
                    codes[at][:first] = e4m3(codes[at][:first] * (old / scale))
                    codes[at][first:hi - j * page] = e4m3(part / scale)
                scales[at] = scale


def attend(q, k_codes, v_codes, k_scales, v_scales, table, lens, cu, scale, causal, window):
    """(out, lse, out magnitude, score magnitude) in float64 for q [tokens, heads, dim].

    The magnitudes are sum_j p_j |v_j| and the largest sum_i |q_i k_ij| * scale of the row.
    """
    tokens, heads, dim = q.shape
    kv_heads, page = k_codes.shape[1], k_codes.shape[2]
    out = np.zeros((tokens, heads, dim))
    size = np.zeros((tokens, heads, dim))
    lse = np.full((tokens, heads), -np.inf)
    reach = np.zeros((tokens, heads))
    for b, length in enumerate(lens):
        n = cu[b + 1] - cu[b]
        ids = [table[b][j] for j in range(-(-length // page))]
        for h in range(heads):
            g = h // (heads // kv_heads)
            if not ids:
                continue
            k = np.concatenate([k_codes[i, g] * float(k_scales[i, g]) for i in ids])[:length]
            v = np.concatenate([v_codes[i, g] * float(v_scales[i, g]) for i in ids])[:length]
            for i in range(n):
                pos = length - n + i
                lo = max(0, pos - window + 1) if window else 0
                hi = min(length, pos + 1) if causal else length
                if hi <= lo:
                    continue
                row = q[cu[b] + i, h].astype(np.float64)
                s = k[lo:hi] @ row * scale
                top = s.max()
                e = np.exp(s - top)
                total = e.sum()
                p = e / total
                out[cu[b] + i, h] = p @ v[lo:hi]
                size[cu[b] + i, h] = p @ np.abs(v[lo:hi])
                lse[cu[b] + i, h] = top + np.log(total)
                reach[cu[b] + i, h] = (np.abs(k[lo:hi]) @ np.abs(row)).max() * abs(scale)
    return out, lse, size, reach
