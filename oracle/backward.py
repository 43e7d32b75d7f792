"""CPU oracle of the MoE block's training pass: the layer norm and the gradients of the layer's
steps.  TEST INFRASTRUCTURE ONLY (see ``oracle.moe``).

Plain float64 numpy, written from the definitions.  Nothing is rounded here: the storage
roundings of the library (h, dg and du in the layer's dtype, each output once) are accounted for by
the tests' tolerances.  Every gradient is pinned to central differences of the forward functions
of ``oracle.moe`` by ``tests/test_backward_oracle.py``.
"""
from __future__ import annotations

from typing import Callable, Dict

import numpy as np

from .moe import decode, expert_matrices

__all__ = ["layer_norm", "layer_norm_backward", "combine_backward", "permute_backward",
           "route_backward", "swiglu_ffn_backward", "grouped_swiglu_backward"]


def layer_norm(x, gamma, beta, eps):
    """(y, mean, rstd) of y[t] = (x[t] - mean_t) * rstd_t * gamma + beta."""
    x = decode(x).astype(np.float64)
    mean = x.mean(axis=1)
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    b = 0.0 if beta is None else np.asarray(beta, np.float64)
    return c * rstd[:, None] * np.asarray(gamma, np.float64) + b, mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta) of layer_norm, with the statistics given."""
    dy, x = decode(dy).astype(np.float64), decode(x).astype(np.float64)
    xh = (x - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    a = dy * np.asarray(gamma, np.float64)
    along = (a * xh).mean(axis=1)[:, None]
    dx = np.asarray(rstd, np.float64)[:, None] * (a - a.mean(axis=1)[:, None] - xh * along)
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def combine_backward(dy, y_perm, row_of, w, k):
    """(dy_perm, dw) of combine: y[t] = sum_j w[t, j] y_perm[row_of[t k + j]]."""
    dy, yp, w = decode(dy).astype(np.float64), np.asarray(y_perm, np.float64), np.asarray(w, np.float64)
    T = w.shape[0]
    dyp, dw = np.zeros_like(yp), np.zeros_like(w)
    for t in range(T):
        for j in range(k):
            r = row_of[t * k + j]
            dyp[r] = w[t, j] * dy[t]
            dw[t, j] = float(dy[t] @ yp[r])
    return dyp, dw


def permute_backward(dx_perm, row_of, k):
    """dx[t] = sum_j dx_perm[row_of[t k + j]]."""
    d = decode(dx_perm).astype(np.float64)
    return d[np.asarray(row_of)].reshape(-1, k, d.shape[1]).sum(axis=1)


def route_backward(idx, w, dw, E):
    """dlogits of the softmax over the chosen experts: its Jacobian diag(w) - w w^T per token."""
    idx, w, dw = np.asarray(idx), np.asarray(w, np.float64), np.asarray(dw, np.float64)
    dl = np.zeros((idx.shape[0], E))
    for t in range(idx.shape[0]):
        g = (np.diag(w[t]) - np.outer(w[t], w[t])) @ dw[t]
        np.add.at(dl[t], idx[t], g)
    return dl


def swiglu_ffn_backward(x, dy, wg, wu, wd):
    """(dx, dwg, dwu, dwd) of y = (silu(x Wg^T) * (x Wu^T)) Wd^T for one expert's rows, and the
    intermediate values by name."""
    x, dy = decode(x).astype(np.float64), decode(dy).astype(np.float64)
    g, u = x @ wg.T, x @ wu.T
    s = 1.0 / (1.0 + np.exp(-g))
    dh = dy @ wd
    h = g * s * u
    du = dh * g * s
    dg = dh * u * s * (1.0 + g * (1.0 - s))
    mid = dict(g=g, u=u, s=s, dh=dh, h=h, du=du, dg=dg)
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ h, mid


def grouped_swiglu_backward(x_perm, dy_perm, offsets, weights_of: Callable[[int], np.ndarray], H: int,
                            I: int) -> Dict[str, np.ndarray]:
    """dx_perm [R, H] and dw [E, 3 H I] (the expert block's layout; zeros for an expert without
    rows)."""
    xp, dyp = decode(x_perm).astype(np.float64), decode(dy_perm).astype(np.float64)
    E = len(offsets) - 1
    dx, dw = np.zeros((xp.shape[0], H)), np.zeros((E, 3 * H * I))
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        d, dwg, dwu, dwd, _ = swiglu_ffn_backward(xp[lo:hi], dyp[lo:hi],
                                                  *expert_matrices(weights_of(e), H, I))
        dx[lo:hi] = d
        dw[e] = np.concatenate([dwg.ravel(), dwu.ravel(), dwd.ravel()])
    return dict(dx_perm=dx, dw=dw)
