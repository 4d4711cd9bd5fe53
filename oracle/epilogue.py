"""64-bit forms of the operators around a layer's products: activations and
their slopes, dropout's generator, and the linear cross-entropy."""
from __future__ import annotations

import math

import numpy as np

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_erf = np.vectorize(math.erf, otypes=[np.float64])


def philox4x32_10(counter, key):
    """Ten rounds of Philox4x32 (Salmon et al., SC'11) on arrays of four
    32-bit counter words and two key words."""
    c = [np.asarray(x, dtype=np.uint64) for x in counter]
    k = [int(key[0]), int(key[1])]
    low, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def keep_mask(rows, cols, p, seed, offset):
    """(elements that stay, their scale, an fp32 number) of dropout over
    [rows x cols]."""
    thr = math.floor(65536 * p + 0.5)
    seed, offset = seed % 2**64, offset % 2**64
    n8 = (cols + 7) // 8
    c0 = np.broadcast_to(np.arange(n8, dtype=np.uint64), (rows, n8))
    c1 = np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, n8))
    full = np.zeros((rows, n8), dtype=np.uint64)
    words = philox4x32_10([c0, c1, full + np.uint64(offset & 0xFFFFFFFF), full + np.uint64(offset >> 32)],
                          (seed & 0xFFFFFFFF, seed >> 32))
    bits = np.empty((rows, n8, 8), dtype=np.uint32)
    for j, w in enumerate(words):
        bits[:, :, 2 * j] = w & np.uint64(0xFFFF)
        bits[:, :, 2 * j + 1] = w >> np.uint64(16)
    return bits.reshape(rows, 8 * n8)[:, :cols] >= thr, (
        float(np.float32(65536 / (65536 - thr))) if thr < 65536 else 0.0)


def drop(x, p, seed, offset):
    keep, scale = keep_mask(x.shape[0], x.shape[1], p, seed, offset)
    return np.where(keep, x * scale, 0.0) if p > 0 else x


def act(z, name):
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name == "gelu":
        return 0.5 * z * (1 + _erf(z / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)))
    if name == "silu":
        return z / (1 + np.exp(-z))
    return z


def slope(z, name):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return 0.5 * (1 + _erf(z / math.sqrt(2))) + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z**3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + np.exp(-z))
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def linear_ce(X, W, labels, keep=None, grad_scale=1.0):
    """X [T x K], W [K x V] in 64 bits -> dict of token_loss, lse, loss, n, P
    (the logits' gradient), dX and dW.  Rows that do not count are not read."""
    T, V = X.shape[0], W.shape[1]
    counted = (labels >= 0) & (labels < V)
    if keep is not None:
        counted &= keep != 0
    rows = np.nonzero(counted)[0]
    n = len(rows)
    z = X[rows] @ W
    top = z.max(axis=1) if n else np.zeros(0)
    e = np.exp(z - top[:, None])
    total = e.sum(axis=1)
    out = {"n": n, "token_loss": np.zeros(T), "lse": np.zeros(T), "dX": np.zeros_like(X),
           "counted": counted}
    y = labels[rows]
    out["lse"][rows] = top + np.log(total)
    out["token_loss"][rows] = out["lse"][rows] - z[np.arange(n), y]
    out["loss"] = out["token_loss"].sum() / max(n, 1)
    P = e / total[:, None] if n else e
    P[np.arange(n), y] -= 1
    P *= grad_scale / max(n, 1)
    out["P"], out["z"] = P, z
    out["dX"][rows] = P @ W.T
    out["dW"] = X[rows].T @ P
    return out
