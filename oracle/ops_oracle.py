"""fp64 NumPy oracle of the operators around the loss: embedding lookup and gradient, 8-bit
activation checkpoints, RMS norm with an 8-bit checkpoint of its input, and the weight gradient
from a checkpoint. Test infrastructure only; written from the definitions in include/ckl.h and
sharing no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

LIMIT = {"int8": 127.0, "e4m3": 448.0}


def embed(ids, W, mask=None, scale=1.0, v0=0):
    """scale * W[ids - v0]; zeros for masked tokens and ids of other rows."""
    ids = np.asarray(ids, np.int64).reshape(-1)
    W = np.asarray(W, np.float64)
    out = np.zeros((len(ids), W.shape[1]))
    for t, v in enumerate(ids):
        if (mask is None or mask[t]) and v0 <= v < v0 + len(W):
            out[t] = float(scale) * W[v - v0]
    return out


def embed_grad(ids, dX, V, mask=None, scale=1.0, v0=0, base=None):
    """(dW, bound): the gradient, and per element the sum of the magnitudes that enter it."""
    dX = np.asarray(dX, np.float64)
    ids = np.asarray(ids, np.int64).reshape(-1)
    dW = np.zeros((V, dX.shape[1])) if base is None else np.array(base, np.float64)
    mag = np.abs(dW)
    for t, v in enumerate(ids):
        if (mask is None or mask[t]) and v0 <= v < v0 + V:
            dW[v - v0] += float(scale) * dX[t]
            mag[v - v0] += abs(float(scale)) * np.abs(dX[t])
    return dW, mag


def e4m3_table():
    """The 256 values of the codes (3 fraction bits, bias 7, no infinities, 0x7F a NaN)."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if c & 127 == 127 else (-v if c & 128 else v)
    return out


def act8_values(q, scale, fmt):
    """The values that codes (uint8, T x cols) and scale bytes (T x blocks) stand for."""
    q = np.asarray(q, np.uint8)
    code = q.view(np.int8).astype(np.float64) if fmt == "int8" else e4m3_table()[q]
    byte = np.repeat(np.asarray(scale, np.int64), 32, axis=1)[:, :q.shape[1]]
    return np.where(byte == 255, np.nan, code * 2.0 ** (byte - 127.0))


def act8_pack(x, fmt):
    """(codes, scale bytes) of x, element by element from the definition."""
    x = np.asarray(x, np.float64)
    T, d = x.shape
    nb = (d + 31) // 32
    q, byte = np.zeros((T, d), np.uint8), np.zeros((T, nb), np.uint8)
    table = e4m3_table()[:127]  # the non-negative codes, ascending
    with np.errstate(invalid="ignore"):
        for t in range(T):
            for b in range(nb):
                v = x[t, 32 * b:32 * b + 32]
                if not np.all(np.isfinite(v)):
                    byte[t, b] = 255
                    continue
                e = -126
                while np.max(np.abs(v)) > LIMIT[fmt] * 2.0 ** e:
                    e += 1
                byte[t, b] = e + 127
                u = v / 2.0 ** e
                if fmt == "int8" and e == 122:  # 64 * 2^122 is no finite float
                    u = np.clip(u, -63, 63)
                if fmt == "e4m3" and e == 120:  # nor is 256 * 2^120
                    u = np.clip(u, -240, 240)
                if fmt == "int8":
                    c = np.round(u).astype(np.int8).view(np.uint8)
                else:
                    hi = np.clip(np.searchsorted(table, np.abs(u)), 0, 126)
                    lo = np.maximum(hi - 1, 0)
                    dl, dh = np.abs(u) - table[lo], table[hi] - np.abs(u)
                    near = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
                    c = (near | np.where(np.signbit(u), 128, 0)).astype(np.uint8)
                q[t, 32 * b:32 * b + 32] = c
    return q, byte


def norm(s, gain, eps):
    """(y, rstd) of the kept sum s."""
    s = np.asarray(s, np.float64)
    rstd = 1.0 / np.sqrt((s * s).mean(1) + float(np.float32(eps)))
    return s * rstd[:, None] * np.asarray(gain, np.float64), rstd


def norm_bwd(dY, kept, rstd, gain, d_sum=None):
    """(dX, dgain, magX, magG) from the checkpoint's values `kept`; mag*: the magnitudes that
    enter each element, for error bounds."""
    dY, kept, g = (np.asarray(a, np.float64) for a in (dY, kept, gain))
    r = np.asarray(rstd, np.float64)[:, None]
    h, a = kept * r, dY * g
    p = 0.0 if d_sum is None else np.asarray(d_sum, np.float64)
    dX = r * (a - h * (a * h).mean(1, keepdims=True)) + p
    mag = r * (np.abs(a) + np.abs(h) * np.abs(a * h).mean(1, keepdims=True)) + np.abs(p)
    return dX, (dY * h).sum(0), mag, np.abs(dY * h).sum(0)


def weight_grad(dY, kept, base=None):
    """(dY^T kept (+ base), magnitudes)."""
    dY, kept = np.asarray(dY, np.float64), np.asarray(kept, np.float64)
    b = 0.0 if base is None else np.asarray(base, np.float64)
    return dY.T @ kept + b, np.abs(dY).T @ np.abs(kept) + np.abs(b)
