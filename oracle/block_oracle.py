"""The operators around the layer, defined in fp64 (numpy): the norm with the
residual add and dropout in front of it, its backward pass, counter-based
dropout, rows quantised to 8 bits and products of such rows.  Written from the
formulas; shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np

MASK32 = (1 << 32) - 1


def philox4x32(counter, key, rounds: int = 10):
    """One Philox4x32 block: four counter words, two key words -> four words
    (Salmon, Moraes, Dror, Shaw, SC 2011), in Python integers."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        hi0, lo0 = divmod(c[0] * 0xD2511F53, 1 << 32)
        hi1, lo1 = divmod(c[2] * 0xCD9E8D57, 1 << 32)
        c = [hi1 ^ c[1] ^ k[0], lo1, hi0 ^ c[3] ^ k[1], lo0]
        k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
    return c


def dropout_draws(T: int, D: int, seed: int, offset: int, site: int) -> np.ndarray:
    """The 16-bit draw of every element of a [T][D] tensor."""
    G = (D + 7) // 8
    hi = (offset + site) % (1 << 64)
    key = (seed & MASK32, (seed >> 32) & MASK32)
    out = np.empty((T * G, 8), dtype=np.int64)
    # vectorised over the groups; one group of the result is checked against
    # philox4x32 by the tests
    n = np.arange(T * G, dtype=np.uint64)
    c = [n & np.uint64(MASK32), n >> np.uint64(32),
         np.full_like(n, hi & MASK32), np.full_like(n, hi >> 32)]
    k = list(key)
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & np.uint64(MASK32),
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & np.uint64(MASK32)]
        k = [(k[0] + 0x9E3779B9) & MASK32, (k[1] + 0xBB67AE85) & MASK32]
    for j in range(4):
        out[:, 2 * j] = (c[j] & np.uint64(0xFFFF)).astype(np.int64)
        out[:, 2 * j + 1] = (c[j] >> np.uint64(16)).astype(np.int64)
    return out.reshape(T, G * 8)[:, :D]


def dropout_factors(T: int, D: int, p: float, seed: int, offset: int, site: int) -> np.ndarray:
    """0 where an element is dropped, else 1 / (probability of being kept)."""
    thr = int(np.floor(p * 65536 + 0.5))
    if thr == 0:
        return np.ones((T, D))
    if thr >= 65536:
        return np.zeros((T, D))
    return np.where(dropout_draws(T, D, seed, offset, site) >= thr, 65536.0 / (65536 - thr), 0.0)


def norm_fwd(s, weight=None, bias=None, eps: float = 1e-5, rms: bool = False):
    """y, mean, rstd of a norm over the rows of s."""
    s = np.asarray(s, dtype=np.float64)
    mean = np.zeros(s.shape[0]) if rms else s.mean(axis=1)
    c = s - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    y = c * rstd[:, None]
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    return y, mean, rstd


def norm_bwd(dy, s, mean, rstd, weight=None, rms: bool = False):
    """ds (without the gradient along the residual), dw, db."""
    dy, s = np.asarray(dy, dtype=np.float64), np.asarray(s, dtype=np.float64)
    mean = np.zeros(s.shape[0]) if rms else np.asarray(mean, dtype=np.float64)
    rstd = np.asarray(rstd, dtype=np.float64)[:, None]
    xhat = (s - mean[:, None]) * rstd
    gw = dy if weight is None else dy * np.asarray(weight, dtype=np.float64)
    ds = gw - xhat * (gw * xhat).mean(axis=1, keepdims=True)
    if not rms:
        ds = ds - gw.mean(axis=1, keepdims=True)
    return ds * rstd, (dy * xhat).sum(axis=0), dy.sum(axis=0)


def quant_rows(x):
    """int8 rows and their fp32 scales; x fp32 (bf16 values widened)."""
    x = np.asarray(x, dtype=np.float32)
    T, D = x.shape
    q = np.zeros((T, D), dtype=np.int8)
    with np.errstate(all="ignore"):
        scale = (np.max(np.abs(x), axis=1) / np.float32(127)).astype(np.float32)
        for t in range(T):
            if np.isfinite(scale[t]) and scale[t] > 0:
                r = np.rint(x[t].astype(np.float64) / np.float64(scale[t]))
                q[t] = np.clip(r, -127, 127).astype(np.int8)
    return q, scale


def matmul_i8(a, a_scale, b, b_scale):
    """y[t][n] = a_scale[t] b_scale[n] sum_k a[t][k] b[n][k]."""
    acc = np.asarray(a, dtype=np.float64) @ np.asarray(b, dtype=np.float64).T
    with np.errstate(invalid="ignore", over="ignore"):
        return (acc * np.asarray(a_scale, dtype=np.float64)[:, None]
                * np.asarray(b_scale, dtype=np.float64)[None, :])
