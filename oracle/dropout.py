"""Dropout from a counter-based generator, and the linear layer with dropout on its
adapter's input, in Python integers and float64.  TEST INFRASTRUCTURE ONLY (see package
docstring).

[TT]'s adapter configuration sets lora_dropout = 0.05; the pages do not say more.
Reading: inverted dropout of the adapter's input alone (the frozen path sees all of X),
with 16 random bits per element from Philox4x32-7 (Salmon et al., 2011), key = seed,
counter = offset + element / 8; kept where the bits reach t = rint(65536 p), kept values
times 65536 / (65536 - t).
"""
from __future__ import annotations

import numpy as np

MULT = (0xD2511F53, 0xCD9E8D57)
WEYL = (0x9E3779B9, 0xBB67AE85)


def philox4x32(counter, key, rounds):
    """The generator's definition: four 32-bit words for a 4-word counter, 2-word key."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        p0, p1 = MULT[0] * c[0], MULT[1] * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + WEYL[0]) & 0xFFFFFFFF, (k[1] + WEYL[1]) & 0xFFFFFFFF]
    return c


def threshold(p):
    return int(np.rint(p * 65536))


def keep(seed, offset, n, p):
    """Which of n elements stay: a bool array."""
    count = (np.arange(-(-n // 8), dtype=np.uint64) + np.uint64(offset % 2 ** 64))
    c = [count & np.uint64(0xFFFFFFFF), count >> np.uint64(32), np.zeros_like(count), np.zeros_like(count)]
    k = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
    low, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(7):
        p0, p1 = np.uint64(MULT[0]) * c[0], np.uint64(MULT[1]) * c[2]
        c = [(p1 >> s) ^ c[1] ^ np.uint64(k[0]), p1 & low, (p0 >> s) ^ c[3] ^ np.uint64(k[1]), p0 & low]
        k = [(k[0] + WEYL[0]) & 0xFFFFFFFF, (k[1] + WEYL[1]) & 0xFFFFFFFF]
    bits = np.empty((len(count), 8), np.uint64)
    for j in range(4):
        bits[:, 2 * j], bits[:, 2 * j + 1] = c[j] & np.uint64(0xFFFF), c[j] >> np.uint64(16)
    return bits.reshape(-1)[:n] >= np.uint64(threshold(p))


def scale(p):
    return 65536.0 / (65536.0 - threshold(p))


def linear_fwd_dropout(W, X, L1, L2, s, p, kept):
    """(Y, T): T = (kept * X)·L1 without the scale; W is h x o, kept M x h."""
    T = np.where(kept, X, 0.0) @ L1
    return X @ W + s * scale(p) * (T @ L2), T


def linear_bwd_dropout(W, X, T, dY, L1, L2, s, p, kept):
    """(dX, dL1, dL2) for the T that the forward gave."""
    q = s * scale(p)
    U = dY @ L2.T
    return (dY @ W.T + q * np.where(kept, U @ L1.T, 0.0), q * (np.where(kept, X, 0.0).T @ U), q * (T.T @ dY))
