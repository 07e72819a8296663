"""fp64 definitions of the operators around the layer: the router's balance loss and its
gradient, one AdamW step (states in 32 or 8 bits), and the adapters of many requests.

Plain NumPy, written from the formulas; shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

BLOCK = 256


def softmax(x):
    x = np.asarray(x, dtype=np.float64)
    top = x.max(axis=-1, keepdims=True)
    z = np.where(np.isneginf(x), 0.0, np.exp(x - np.where(np.isneginf(top), 0.0, top)))
    s = z.sum(axis=-1, keepdims=True)
    return np.divide(z, s, out=np.zeros_like(z), where=s != 0)   # a row of -inf: zeros


def _rows(T, offsets, mask, s):
    """Valid rows of sequence s."""
    lo, hi = (0, T) if offsets is None else (int(offsets[s]), int(offsets[s + 1]))
    rows = np.arange(lo, hi)
    return rows if mask is None else rows[np.asarray(mask)[lo:hi] != 0]


def balance_loss(logits, ids, S=1, offsets=None, mask=None):
    """(loss [S], counts [S, E], n [S])."""
    T, E = logits.shape
    k = ids.shape[1]
    loss, counts, n = np.zeros(S), np.zeros((S, E), dtype=np.int64), np.zeros(S, dtype=np.int64)
    for s in range(S):
        rows = _rows(T, offsets, mask, s)
        n[s] = len(rows)
        if len(rows) == 0:
            continue
        counts[s] = np.bincount(ids[rows].ravel(), minlength=E)
        f = counts[s] / (k * len(rows))
        loss[s] = E * np.sum(f * softmax(logits[rows]).mean(axis=0))
    return loss, counts, n


def balance_backward(logits, counts, n, dloss, k, offsets=None, mask=None):
    """dlogits [T, E] with the counts held constant."""
    T, E = logits.shape
    out = np.zeros((T, E))
    for s in range(len(n)):
        rows = _rows(T, offsets, mask, s)
        if len(rows) == 0:
            continue
        p = softmax(logits[rows])
        f = counts[s] / (k * len(rows))
        out[rows] = dloss[s] * E / len(rows) * p * (f - (p * f).sum(axis=1, keepdims=True))
    return out


def adamw(w, g, m, v, t, lr, b1, b2, eps, wd):
    """(w, m, v) after step t (counted from 1)."""
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    w = w * (1 - lr * wd) - lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return w, m, v


# ---- 8-bit states: e4m3 values times a block scale
def e4m3_values():
    """The values of codes 0x00 .. 0x7E."""
    c = np.arange(0x7F)
    e, f = c >> 3, c & 7
    return np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7.0))


def decode(codes, scales):
    codes = np.asarray(codes, dtype=np.int64)
    sign = np.where(codes & 0x80, -1.0, 1.0)
    return sign * e4m3_values()[codes & 0x7F] * np.repeat(np.asarray(scales, dtype=np.float64), BLOCK)


def mix32(x):
    x = np.asarray(x, dtype=np.uint64) & np.uint64(0xFFFFFFFF)
    for shift, mul in ((16, 0x9E3779B9), (15, 0xBB67AE85)):
        x = ((x ^ (x >> np.uint64(shift))) * np.uint64(mul)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def noise(t, n):
    """The two 16-bit random numbers of each element at step t, as fractions."""
    h = mix32(np.arange(n, dtype=np.uint64) ^ mix32(t))
    return (h & np.uint64(0xFFFF)) / 65536.0, (h >> np.uint64(16)) / 65536.0


def encode(x, u, least_one=False):
    """(codes, scales, place) of x padded to whole blocks: the code below |x| / scale, plus one
    where `place`, the way to the next code plus u, reaches one."""
    pad = -len(x) % BLOCK
    x, u = np.pad(x, (0, pad)), np.pad(u, (0, pad))
    top = np.abs(x.reshape(-1, BLOCK)).max(axis=1)
    top = np.where(top < 2.0 ** -100, 0.0, top)
    scales = top / 448
    big = np.repeat(top, BLOCK)
    y = np.divide(np.abs(x) * 448, big, out=np.zeros_like(x), where=big > 0)
    vals = e4m3_values()
    below = np.searchsorted(vals, y, side="right") - 1
    nxt = vals[np.minimum(below + 1, 0x7E)]
    gap = np.where(nxt > vals[below], nxt - vals[below], 32.0)
    place = (y - vals[below]) / gap + u
    codes = np.minimum(below + (place >= 1), 0x7E)
    if least_one:
        codes = np.where((x > 0) & (big > 0) & (codes == 0), 1, codes)
    codes = np.where((x < 0) & (codes > 0), codes | 0x80, codes)
    return codes, scales, place


def lora_requests(X, adapters, A, B, scale, Y, offsets=None):
    """Y with scale (X A) B added to the rows of every request with an adapter."""
    Y = np.array(Y, dtype=np.float64)
    for s, a in enumerate(adapters):
        lo, hi = (s, s + 1) if offsets is None else (int(offsets[s]), int(offsets[s + 1]))
        if a >= 0 and hi > lo:
            Y[lo:hi] += scale[a] * (X[lo:hi] @ A[a]) @ B[a]
    return Y
