"""fp64 oracle of the routing rules and the 8-bit integer operators: plain numpy, row by
row where order matters. Test infrastructure only; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def scores(row, score):
    """Scores of one row of logits; experts that are off (-inf, NaN) have 0."""
    x = np.asarray(row, dtype=np.float64)
    on = ~(np.isnan(x) | (x == -np.inf))
    x = np.where(on, np.minimum(x, np.finfo(np.float32).max), 0.0)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s = np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
    else:
        e = np.exp(x - (x[on].max() if on.any() else 0.0))
        s = e / max(e[on].sum(), 1e-300)
    return np.where(on, s, 0.0), on


def choose(row, k, score, bias=None, groups=1, top_groups=1, group_top=2):
    """The k chosen experts. A bias of NaN counts as -inf, one of +inf as the largest finite fp32 value; a key of
    -inf ranks below all others and adds nothing to its group."""
    x = np.asarray(row, dtype=np.float64)
    if bias is not None:
        bias = np.asarray(bias, np.float64)
        bias = np.where(np.isnan(bias), -np.inf, np.minimum(bias, np.finfo(np.float32).max))
    E = len(x)
    s, on = scores(row, score)
    if bias is None and (groups == 1 or top_groups == groups):
        key = np.where(on, x, -np.inf)
    else:
        key = np.where(on, s + (0.0 if bias is None else bias), -np.inf)
    left = list(range(E))
    if groups > 1 and top_groups < groups:
        per = E // groups
        total = []
        for g in range(groups):
            best = sorted(key[g * per:(g + 1) * per], reverse=True)[:group_top]
            best = [b for b in best if b != -np.inf]
            total.append(sum(best) if best else -np.inf)
        kept = sorted(range(groups), key=lambda g: (-total[g], g))[:top_groups]
        left = [e for e in left if e // per in kept]
    return sorted(left, key=lambda e: (-key[e], e))[:k]


def ratios(row, idx, score):
    """Scores of the chosen over their sum, taken on their logarithms: scores too small for any
    number format still have ratios. 0 for experts that are off."""
    _, on = scores(row, score)
    x, on = np.asarray(row, dtype=np.float64)[list(idx)], on[list(idx)]
    if not on.any():
        return np.zeros(len(idx))
    x = np.where(on, np.minimum(x, np.finfo(np.float32).max), 0.0)
    log = x if score == "softmax" else np.minimum(x, 0) - np.log1p(np.exp(-np.abs(x)))
    r = np.where(on, np.exp(np.minimum(log - log[on].max(), 0)), 0.0)
    return r / r.sum()


def weights(row, idx, score, renormalise=True, scale=1.0):
    return scale * (ratios(row, idx, score) if renormalise else scores(row, score)[0][list(idx)])


def route(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_top=2, renormalise=True, scale=1.0):
    idx = np.array([choose(r, k, score, bias, groups, top_groups, group_top) for r in logits], dtype=np.int64)
    idx = idx.reshape(len(logits), k)
    w = np.array([weights(r, i, score, renormalise, scale) for r, i in zip(logits, idx)]).reshape(len(logits), k)
    return idx, w


def route_backward(d_w, logits, idx, score="softmax", renormalise=True, scale=1.0):
    """(d_logits, a magnitude that bounds the terms each element is made of)."""
    out, mag = np.zeros(np.shape(logits)), np.zeros(np.shape(logits))
    for t, row in enumerate(logits):
        s, on = scores(row, score)
        i = [e for e in idx[t] if 0 <= e < len(s)]
        d = scale * np.asarray([v for v, e in zip(d_w[t], idx[t]) if 0 <= e < len(s)], np.float64) * on[i]
        # s * d loss / d s of the chosen, and the sum that a softmax takes off every expert
        if renormalise:
            r = ratios(row, i, score)
            a, m = r * (d - (d * r).sum()), r * (np.abs(d) + np.abs(d * r).sum())
        else:
            a, m = s[i] * d, s[i] * np.abs(d)
        if score == "sigmoid":
            out[t, i], mag[t, i] = (1 - s[i]) * a, m
        else:
            out[t, i], mag[t, i] = a, m
            if not renormalise:
                out[t] -= s * a.sum()
                mag[t] += s * m.sum()
    return out, mag


def quantize(x):
    """(q, scale as held in fp32, distance of each quotient from the nearest half) of the rows of x."""
    x = np.asarray(x, dtype=np.float64)
    amax = np.abs(x).max(axis=-1, keepdims=True)
    inv = np.float64(np.float32(1) / np.float32(127))   # both the constant and the product rounded to fp32
    scale = np.where(amax > 0, (amax * inv).astype(np.float32).astype(np.float64), 1.0)
    r = np.divide(x, scale, out=np.zeros_like(x), where=scale > 0)
    q = np.clip(np.rint(r), -127, 127)
    return q, scale[..., 0], np.abs(np.abs(r - np.floor(r)) - 0.5)


def matmul(x, w, w_scale, x_scale=None):
    if x_scale is None:
        q, x_scale, _ = quantize(x)
    else:
        q = np.asarray(x, np.float64)
    return q @ np.asarray(w, np.float64).T * np.asarray(x_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)


#: A quotient nearer to a half than this may be rounded the other way by 32-bit SwiGLU outputs.
UNSURE = 5e-4


def experts(x, idx, w, gate_up, gate_up_scale, down, down_scale):
    """(out, the sum of the terms' magnitudes, what quotients next to a half may change)."""
    T, H = np.shape(x)
    out, mag, unsure = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    I = np.shape(down)[2]
    for t in range(T):
        for j, e in enumerate(idx[t]):
            if e < 0 or e >= len(down):
                continue
            a = matmul(x[t:t + 1], gate_up[e], gate_up_scale[e])[0]
            g, u = a[:I], a[I:]
            h = g / (1 + np.exp(-g)) * u
            q, s, near = quantize(h[None])
            d = np.asarray(down[e], np.float64)
            f = abs(float(w[t, j])) * s[0] * np.asarray(down_scale[e], np.float64)
            out[t] += float(w[t, j]) * s[0] * np.asarray(down_scale[e], np.float64) * (d @ q[0])
            mag[t] += f * (np.abs(d) @ np.abs(q[0]))
            unsure[t] += f * (np.abs(d) @ (near[0] < UNSURE))
    return out, mag, unsure

