"""Softmax cross entropy of an output head, in float64.  TEST INFRASTRUCTURE ONLY (see
package docstring).

[MC] "One training step" and [TT] §4 "One QLoRA Training Step, End to End" name the loss
without writing it out.  Reading: the next-token cross entropy of a linear head, with
z = H·W^T, loss = log(sum exp z) - z[label] per token; a token whose label is no word of
the vocabulary carries none.
"""
from __future__ import annotations

import numpy as np


def loss_fwd(H, W, labels):
    """(loss, lse) per token; 0 for the tokens without a loss."""
    V = W.shape[0]
    loss, lse = np.zeros(len(labels)), np.zeros(len(labels))
    for i, y in enumerate(labels):
        if 0 <= y < V:
            z = W.astype(np.float64) @ H[i].astype(np.float64)
            lse[i] = z.max() + np.log(np.sum(np.exp(z - z.max())))
            loss[i] = lse[i] - z[y]
    return loss, lse


def loss_grad(H, W, labels, dloss):
    """G = dloss * d loss / d z, [tokens][V]."""
    V = W.shape[0]
    G = np.zeros((len(labels), V))
    for i, y in enumerate(labels):
        if 0 <= y < V:
            z = W.astype(np.float64) @ H[i].astype(np.float64)
            e = np.exp(z - z.max())
            G[i] = dloss[i] * e / e.sum()
            G[i, y] -= dloss[i]
    return G


def loss_bwd(H, W, labels, dloss):
    """(dH, dW) for the gradient dloss of each token's loss."""
    G = loss_grad(H, W, labels, dloss)
    live = [i for i, y in enumerate(labels) if 0 <= y < W.shape[0]]
    return G @ W.astype(np.float64), G[live].T @ H[live].astype(np.float64)
