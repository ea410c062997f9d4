"""float64 oracle of the expert-grouped linear and of counter-based dropout
(test infrastructure only).

Dropout keeps element i of a tensor where 16-bit half i % 8 of the Philox4x32
block (10 rounds; J. Salmon, M. Moraes, R. Dror, D. Shaw, "Parallel random
numbers: as easy as 1, 2, 3", SC'11) of counter offset + i // 8 under the key
`seed` is at least t = floor(p 2^16 + 1/2), and scales what it keeps by
2^16 / (2^16 - t).

The grouped layer is the dense one (oracle/linear.py) of each expert on its own
rows, its adapter branch reading D(X).
"""
from __future__ import annotations

import math

import numpy as np


def philox4x32_10(counter: np.ndarray, key: int) -> np.ndarray:
    """Words [n, 4] (uint32) of the 64-bit counters [n] (upper counter words 0)."""
    mask = np.uint64(0xFFFFFFFF)
    counter = np.asarray(counter, np.uint64)
    c = [counter & mask, counter >> np.uint64(32), np.zeros_like(counter), np.zeros_like(counter)]
    return _rounds(c, key & 0xFFFFFFFF, (key >> 32) & 0xFFFFFFFF)


def _rounds(c, k0: int, k1: int) -> np.ndarray:
    mask, hi = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        with np.errstate(over="ignore"):
            a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> hi) ^ c[1] ^ np.uint64(k0), b & mask, (a >> hi) ^ c[3] ^ np.uint64(k1), a & mask]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, 1).astype(np.uint32)


def threshold(p: float) -> int:
    return int(math.floor(p * 65536.0 + 0.5))


def factor(p: float) -> float:
    return 65536.0 / (65536.0 - threshold(p))


def keep_mask(n: int, p: float, seed: int, offset: int = 0, first: int = 0) -> np.ndarray:
    """Truth values of elements first .. first + n - 1 (first % 8 == 0)."""
    assert first % 8 == 0
    groups = (n + 7) // 8
    counters = (np.arange(groups, dtype=np.uint64) + np.uint64((offset + first // 8) % 2**64))
    words = philox4x32_10(counters, seed)
    return words.astype("<u4").view("<u2").reshape(-1)[:n] >= threshold(p)


def dropout(x: np.ndarray, p: float, seed: int, offset: int = 0) -> np.ndarray:
    keep = keep_mask(x.size, p, seed, offset).reshape(x.shape)
    return np.where(keep, x * factor(p), 0.0)


def grouped_fwd(X, W, offsets, A, B, alpha: float, drop=None):
    """Y [T, N], XA [T, r] (NaN in rows that no expert owns): X [T, K], W [E, N, K], A [E, K, r], B [E, r, N];
    drop = (p, seed, offset) or None."""
    T, r = X.shape[0], A.shape[2]
    s = alpha / r
    D = X if drop is None else dropout(X, *drop)
    Y, XA = np.full((T, W.shape[1]), np.nan), np.full((T, r), np.nan)
    for e in range(len(offsets) - 1):
        rows = slice(offsets[e], offsets[e + 1])
        XA[rows] = D[rows] @ A[e]
        Y[rows] = X[rows] @ W[e].T + s * (XA[rows] @ B[e])
    return Y, XA


def grouped_bwd(X, dY, W, offsets, A, B, alpha: float, XA=None, drop=None):
    """dX [T, K] (NaN in rows that no expert owns), dA, dB."""
    r = A.shape[2]
    s = alpha / r
    D = X if drop is None else dropout(X, *drop)
    M = np.ones_like(X) if drop is None else dropout(np.ones_like(X), *drop)
    dX, dA, dB = np.full(X.shape, np.nan), np.zeros_like(A), np.zeros_like(B)
    for e in range(len(offsets) - 1):
        rows = slice(offsets[e], offsets[e + 1])
        xa = D[rows] @ A[e] if XA is None else XA[rows]
        G = s * (dY[rows] @ B[e].T)
        dX[rows] = dY[rows] @ W[e] + M[rows] * (G @ A[e].T)
        dA[e] = D[rows].T @ G
        dB[e] = s * (xa.T @ dY[rows])
    return dX, dA, dB
