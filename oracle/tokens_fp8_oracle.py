"""fp64 oracle of token dispatch and combine and of the 8-bit floating-point operators: plain
numpy. Test infrastructure only; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np

BLOCK = 128


def _e4m3_table():
    """The value of each E4M3 code: sign, 4 bits of exponent (bias 7), 3 of mantissa; 0x7F and 0xFF are NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[c] = np.nan if c & 127 == 127 else -v if c & 128 else v
    return out


E4M3 = _e4m3_table()
_POSITIVE = E4M3[:127]


def to_e4m3(v):
    """Codes of the nearest values, halves to the even code, held to +-448; NaN is 0x7F."""
    a = np.minimum(np.abs(np.asarray(v, np.float64)), 448.0)
    hi = np.clip(np.searchsorted(_POSITIVE, np.nan_to_num(a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(np.signbit(v), code | 128, code)
    return np.where(np.isnan(v), 127, code).astype(np.uint8)


def quantize(x):
    """(codes [T, K], scales [T, blocks]) of rows: scale and quotient held in 32 bits."""
    x = np.asarray(x, np.float64)
    T, K = x.shape
    n = -(-K // BLOCK)
    codes, scales = np.empty((T, K), np.uint8), np.empty((T, n), np.float32)
    for b in range(n):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        amax = np.abs(part).max(axis=1)
        bad = ~np.isfinite(part).all(axis=1)
        with np.errstate(all="ignore"):
            s = np.where(bad, np.float32(np.nan), amax.astype(np.float32) * np.float32(1 / 448))
            s = np.where(s == 0, np.float32(1), s).astype(np.float32)
            codes[:, b * BLOCK:(b + 1) * BLOCK] = to_e4m3((part.astype(np.float32) / s[:, None]).astype(np.float32))
        scales[:, b] = s
    return codes, scales


def swiglu(x):
    g, u = np.split(np.asarray(x, np.float64), 2, axis=1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def matmul(x, x_scale, w, w_scale):
    """(out, the sum of the terms' magnitudes): x [T, K] and w [N, K] values, scales by block."""
    T, K = x.shape
    N = len(w)
    out, mag = np.zeros((T, N)), np.zeros((T, N))
    channel = np.arange(N) // BLOCK
    for b in range(-(-K // BLOCK)):
        at = slice(b * BLOCK, (b + 1) * BLOCK)
        s = np.asarray(x_scale, np.float64)[:, b, None] * np.asarray(w_scale, np.float64)[channel, b]
        out += x[:, at] @ w[:, at].T * s
        mag += np.abs(x[:, at]) @ np.abs(w[:, at]).T * np.abs(s)
    return out, mag


def grouped_matmul(x, x_scale, offsets, w, w_scale):
    out, mag = np.zeros((len(x), w.shape[1])), np.zeros((len(x), w.shape[1]))
    for e in range(len(w)):
        at = slice(offsets[e], offsets[e + 1])
        if at.stop > at.start:
            out[at], mag[at] = matmul(x[at], x_scale[at], w[e], w_scale[e])
    return out, mag


def places(idx, E):
    """(offsets [E + 1], pos [T, k]), one choice after the other."""
    T, k = np.shape(idx)
    lists = [[] for _ in range(E + 1)]
    for a, e in enumerate(np.reshape(idx, -1)):
        lists[e if 0 <= e < E else E].append(a)
    offsets = np.concatenate([[0], np.cumsum([len(v) for v in lists])])[:E + 1]
    pos = np.empty(T * k, np.int64)
    for r, a in enumerate(sum(lists, [])):
        pos[a] = r if r < offsets[E] else ~r
    return offsets, pos.reshape(T, k)


def dispatch(x, pos):
    rows = np.zeros((pos.size, np.shape(x)[1]), np.asarray(x).dtype)
    for t, j in np.ndindex(pos.shape):
        if pos[t, j] >= 0:
            rows[pos[t, j]] = x[t]
    return rows


def combine(y, pos, weights):
    """(out, the sum of the terms' magnitudes)."""
    y, w = np.asarray(y, np.float64), np.asarray(weights, np.float64)
    g = np.where((pos >= 0)[..., None], y[np.maximum(pos, 0)], 0.0) * w[..., None]
    return g.sum(1), np.abs(g).sum(1)


def combine_backward(d_out, y, pos, weights):
    """(d_y, d_weights, the sum of the magnitudes of d_weights' terms)."""
    d, y, w = (np.asarray(v, np.float64) for v in (d_out, y, weights))
    d_y = np.zeros(np.shape(y))
    d_w, mag = np.zeros(pos.shape), np.zeros(pos.shape)
    for t, j in np.ndindex(pos.shape):
        if pos[t, j] >= 0:
            d_y[pos[t, j]] = w[t, j] * d[t]
            d_w[t, j] = (d[t] * y[pos[t, j]]).sum()
            mag[t, j] = np.abs(d[t] * y[pos[t, j]]).sum()
    return d_y, d_w, mag
