"""Norms before and after a transformer block with its gate and residual scale, in
float64.  TEST INFRASTRUCTURE ONLY (see package docstring).

[MC] "A closer look: Design choices and memory costs": the adapted linears sit in the
blocks of a transformer.  Reading: a block's output Y joins the residual stream R, and
the stream is RMS-normalised for the next block; a block may have a norm of its output,
a gate per channel and one scale of its contribution as well.  With
rms(x) = sqrt(mean(x^2) + eps) over a row:
  u = Y or Y / rms(Y) * w_post,   R' = R + alpha * gate * u,   N = R' / rms(R') * w_pre.

Inputs are float arrays holding the exact values of the tensors; nothing is rounded here.
"""
from __future__ import annotations

import numpy as np


def rstd(x, eps):
    x = np.asarray(x, np.float64)
    return 1.0 / np.sqrt(np.mean(x * x, axis=1) + eps)


def norm_fwd(r, y, w_pre, w_post, gate, alpha, eps):
    """(R', N, rstd_pre, rstd_post); y, w_pre, w_post and gate may be None."""
    r = np.asarray(r, np.float64)
    q = None
    if y is not None:
        u = np.asarray(y, np.float64)
        if w_post is not None:
            q = rstd(u, eps)
            u = u * q[:, None] * w_post
        r = r + alpha * (1.0 if gate is None else gate) * u
    if w_pre is None:
        return r, None, None, q
    p = rstd(r, eps)
    return r, r * p[:, None] * w_pre, p, q


def _through_norm(g, x, s):
    """The gradient of x for the gradient g of x * s, s = rstd(x) varying with x:
    d(x_k s)/dx_j = s (k == j) - s^3 x_k x_j / h."""
    h = x.shape[1]
    return s[:, None] * g - (s ** 3 / h * np.sum(g * x, axis=1))[:, None] * x


def norm_bwd(dn, dr_out, r_out, y, rstd_pre, rstd_post, w_pre, w_post, gate, alpha):
    """(dR, dY, dw_pre, dw_post, dgate); what does not apply is None."""
    dr = 0.0 if dr_out is None else np.asarray(dr_out, np.float64)
    dw_pre = dw_post = dgate = None
    if w_pre is not None:
        dr = dr + _through_norm(dn * w_pre, r_out, rstd_pre)
        dw_pre = np.sum(dn * r_out * rstd_pre[:, None], axis=0)
    g = 1.0 if gate is None else gate
    du = alpha * g * dr
    dy, u = du, y
    if w_post is not None:
        dy = _through_norm(du * w_post, y, rstd_post)
        dw_post = np.sum(du * y * rstd_post[:, None], axis=0)
        u = y * rstd_post[:, None] * w_post
    if gate is not None and u is not None:
        dgate = np.sum(alpha * dr * u, axis=0)
    return dr, dy, dw_pre, dw_post, dgate
