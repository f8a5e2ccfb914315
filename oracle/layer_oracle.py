"""Plain CPU oracle of the steps around the experts (test infrastructure only).

NumPy in 64 bits, straight from the definitions in ``include/ultraep_layer.h``:
routing, the norm with the residual, the gated activation, and their gradients.
Shares no code with the HIP path.
"""
from __future__ import annotations

import numpy as np

F32_MAX = float(np.finfo(np.float32).max)


def clean(logits):
    """(masked, logits): -inf and NaN masked, +inf the largest finite fp32."""
    l = np.asarray(logits, dtype=np.float64)
    masked = np.isnan(l) | (l == -np.inf)
    return masked, np.minimum(np.where(masked, 0.0, l), F32_MAX)


def scores(logits, sigmoid: bool):
    masked, l = clean(logits)
    with np.errstate(over="ignore"):
        if sigmoid:
            return np.where(masked, 0.0, 1.0 / (1.0 + np.exp(-l)))
        m = np.where(masked, -np.inf, l).max(axis=1, keepdims=True)
        t = np.where(masked, 0.0, np.exp(np.where(masked, 0.0, l - np.where(np.isfinite(m), m, 0.0))))
    total = t.sum(axis=1, keepdims=True)
    return np.divide(t, total, out=np.zeros_like(t), where=total > 0)


def chosen_weights(logits, idx, sigmoid: bool, renorm: bool, scale: float):
    """Weights of the ids idx [T, k] (none for ids that name no expert, or a masked one)."""
    masked, l = clean(logits)
    s = scores(logits, sigmoid)
    w = np.zeros(idx.shape)
    for t in range(idx.shape[0]):
        js = [j for j, e in enumerate(idx[t]) if 0 <= e < l.shape[1] and not masked[t, e]]
        if not js:
            continue
        es = idx[t, js]
        if not renorm:
            w[t, js] = scale * s[t, es]
            continue
        x = l[t, es]
        with np.errstate(over="ignore"):
            logs = -np.logaddexp(0.0, -x) if sigmoid else x  # of the scores, up to a common term
        p = np.exp(logs - logs.max())
        w[t, js] = scale * p / p.sum()
    return w


def route(logits, k: int, sigmoid=False, bias=None, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0):
    """(idx [T, k], w [T, k])."""
    masked, l = clean(logits)
    T, E = l.shape
    s = scores(logits, sigmoid)
    if bias is None:
        key = np.where(masked, -np.inf, l)
    else:
        b = np.asarray(bias, dtype=np.float64)
        key = np.where(masked | np.isnan(b), -np.inf, s + np.where(np.isnan(b), 0.0, b))
    idx = np.full((T, k), -1, dtype=np.int32)
    per = E // groups
    for t in range(T):
        kt = key[t].copy()
        if groups > 1:
            worth = np.full(groups, -np.inf)
            for g in range(groups):
                part = kt[g * per:(g + 1) * per]
                if group_top == 2:
                    values = s[t, g * per:(g + 1) * per] if bias is None else part
                    best = np.sort(values[part > -np.inf])[::-1][:2]
                    if len(best):
                        worth[g] = best.sum()
                else:
                    worth[g] = part.max()
            order = np.argsort(-worth, kind="stable")[:topk_groups]
            keep = {int(g) for g in order if worth[g] > -np.inf}
            for g in range(groups):
                if g not in keep:
                    kt[g * per:(g + 1) * per] = -np.inf
        order = np.argsort(-kt, kind="stable")[:k]
        order = order[kt[order] > -np.inf]
        idx[t, :len(order)] = order
    return idx, chosen_weights(logits, idx, sigmoid, renorm, scale)


def route_backward(logits, idx, grad_w, sigmoid=False, renorm=True, scale=1.0):
    """(gradients of the logits, sums of the magnitudes that they are made of)."""
    masked, l = clean(logits)
    s = scores(logits, sigmoid)
    w = chosen_weights(logits, idx, sigmoid, renorm, scale)
    out, mag = np.zeros_like(l), np.zeros_like(l)
    for t in range(idx.shape[0]):
        js = [j for j, e in enumerate(idx[t]) if 0 <= e < l.shape[1] and not masked[t, e]]
        total = sum(w[t, j] * grad_w[t, j] for j in js)
        total_mag = sum(abs(w[t, j] * grad_w[t, j]) for j in js)
        if not sigmoid and not renorm:
            out[t], mag[t] = -s[t] * total, s[t] * total_mag
        for j in js:
            e = idx[t, j]
            d, m = w[t, j] * grad_w[t, j], abs(w[t, j] * grad_w[t, j])
            if renorm:
                d, m = d - w[t, j] * total / scale, m + abs(w[t, j] * total_mag / scale)
            if sigmoid:
                d = d * (1.0 - s[t, e])
            out[t, e] += d
            mag[t, e] += m
    return out, mag


def residual_norm(h, weight, eps: float):
    """(rstd, y) of the stream's rows h (the sum as it is stored)."""
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return rstd, h * rstd[:, None] * weight


def residual_norm_backward(grad_y, h, weight, rstd, grad_in=None):
    """(grad_h, its magnitude, grad_weight, its magnitude)."""
    v, z = rstd[:, None], weight * grad_y
    n = h * v
    back = np.zeros_like(h) if grad_in is None else grad_in
    d = back + v * (z - n * np.mean(z * n, axis=1, keepdims=True))
    mag = np.abs(back) + v * (np.abs(z) + np.abs(n) * np.mean(np.abs(z * n), axis=1, keepdims=True))
    return d, mag, (grad_y * n).sum(axis=0), np.abs(grad_y * n).sum(axis=0)


def gate(g, gelu: bool):
    """f(g) = g / (1 + exp(-z)), its derivative, and the magnitude that this is made of."""
    c = 2.0 * np.sqrt(2.0 / np.pi)
    z, dz = (c * (g + 0.044715 * g ** 3), c * (1.0 + 3 * 0.044715 * g * g)) if gelu else (g, np.ones_like(g))
    with np.errstate(over="ignore"):
        p, r = 1.0 / (1.0 + np.exp(-z)), 1.0 / (1.0 + np.exp(z))
    return g * p, p + g * p * r * dz, p + np.abs(g * p * r * dz)


def nothing_tiny(x):
    return np.where(np.abs(x) < 2.0 ** -100, 0.0, x)


def glu(h, gelu=False):
    F = h.shape[1] // 2
    return nothing_tiny(gate(h[:, :F], gelu)[0] * h[:, F:])


def glu_backward(h, grad, gelu=False):
    """(gradient rows, sums of the magnitudes that they are made of)."""
    F = h.shape[1] // 2
    f, df, m = gate(h[:, :F], gelu)
    d = np.concatenate([grad * h[:, F:] * df, grad * f], axis=1)
    return nothing_tiny(d), np.concatenate([np.abs(grad * h[:, F:]) * m, np.abs(grad * f)], axis=1)
