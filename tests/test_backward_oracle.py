"""Pins of the training pass's oracle (``oracle.backward``) to central differences of the forward
functions of ``oracle.moe``, and planted mistakes that those pins must catch (CPU only).

Tolerance: with step h a central difference of a smooth f is off by h^2 |f'''| / 6 plus the
cancellation 2^-52 |f| / h.  At h = 2^-14 (1e-4 below) on values of order one to ten that is a few
1e-8 plus a few 1e-11 times the size of the loss (at most about 1e2 here); 2e-6 leaves two orders
for third derivatives above one.
"""
import os
import sys

import numpy as np
import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from oracle import backward as G  # noqa: E402
from oracle import moe as O  # noqa: E402

STEP, TOL = 2.0 ** -14, 2e-6


def differences(f, x):
    """d f / d x by central differences, element by element (f: array -> number)."""
    x = np.array(x, np.float64)
    out = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        keep = x[i]
        x[i] = keep + STEP
        hi = f(x)
        x[i] = keep - STEP
        lo = f(x)
        x[i] = keep
        out[i] = (hi - lo) / (2 * STEP)
    return out


def pin_layer_norm():
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 5)) + 0.7, rng.standard_normal((3, 5))
    gamma, beta = 1 + 0.3 * rng.standard_normal(5), rng.standard_normal(5)
    eps = 1e-3
    loss = lambda x_, g_, b_: float((dy * G.layer_norm(x_, g_, b_, eps)[0]).sum())
    _, mean, rstd = G.layer_norm(x, gamma, beta, eps)
    dx, dg, db = G.layer_norm_backward(dy, x, gamma, mean, rstd)
    np.testing.assert_allclose(dx, differences(lambda v: loss(v, gamma, beta), x), atol=TOL)
    np.testing.assert_allclose(dg, differences(lambda v: loss(x, v, beta), gamma), atol=TOL)
    np.testing.assert_allclose(db, differences(lambda v: loss(x, gamma, v), beta), atol=TOL)


def _routed(T, E, k, seed):
    rng = np.random.default_rng(seed)
    logits = 2 * rng.standard_normal((T, E))
    idx, w = O.route(logits, k)
    row_of, src_of = O.permutation(idx, E)
    return rng, logits, idx, np.asarray(w, np.float64), row_of, src_of


def _weights(logits, idx):
    z = np.take_along_axis(np.asarray(logits, np.float64), idx.astype(np.int64), 1)
    ex = np.exp(z - z.max(1, keepdims=True))
    return ex / ex.sum(1, keepdims=True)


def pin_combine():
    rng, _, _, w, row_of, _ = _routed(4, 6, 3, 2)
    yp, dy = rng.standard_normal((12, 5)), rng.standard_normal((4, 5))
    dyp, dw = G.combine_backward(dy, yp, row_of, w, 3)
    loss = lambda yp_, w_: float((dy * O.combine(yp_, row_of, w_, 3)).sum())
    np.testing.assert_allclose(dyp, differences(lambda v: loss(v, w), yp), atol=TOL)
    np.testing.assert_allclose(dw, differences(lambda v: loss(yp, v), w), atol=TOL)


def pin_permute():
    rng, _, _, _, row_of, src_of = _routed(4, 6, 3, 3)
    x, d = rng.standard_normal((4, 5)), rng.standard_normal((12, 5))
    loss = lambda x_: float((d * x_[src_of // 3]).sum())
    np.testing.assert_allclose(G.permute_backward(d, row_of, 3), differences(loss, x), atol=TOL)


def pin_route():
    rng, logits, idx, w, _, _ = _routed(4, 7, 3, 4)
    dw = rng.standard_normal((4, 3))
    loss = lambda l_: float((dw * _weights(l_, idx)).sum())
    got = G.route_backward(idx, _weights(logits, idx), dw, 7)
    np.testing.assert_allclose(got, differences(loss, logits), atol=TOL)


def pin_experts():
    rng = np.random.default_rng(5)
    H, I, E = 4, 3, 3
    offsets = np.array([0, 2, 2, 5])
    x, dy = rng.standard_normal((5, H)), rng.standard_normal((5, H))
    w = rng.standard_normal((E, 3 * H * I))

    def loss(x_, w_):
        return float((dy * O.grouped_swiglu(x_, offsets, lambda e: w_[e], H, I, False)).sum())

    got = G.grouped_swiglu_backward(x, dy, offsets, lambda e: w[e], H, I)
    np.testing.assert_allclose(got["dx_perm"], differences(lambda v: loss(v, w), x), atol=TOL)
    np.testing.assert_allclose(got["dw"], differences(lambda v: loss(x, v), w), atol=TOL)
    assert not got["dw"][1].any()


def pin_whole_layer():
    """The chain of the five, as the layer runs it, against differences of the whole layer."""
    rng, logits, idx, _, row_of, src_of = _routed(3, 5, 2, 6)
    T, E, k, H, I = 3, 5, 2, 4, 3
    x, dy = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    gamma, beta = 1 + 0.2 * rng.standard_normal(H), 0.1 * rng.standard_normal(H)
    w = rng.standard_normal((E, 3 * H * I))
    offsets = O.expert_offsets(O.expert_counts(idx, E))
    eps = 1e-3

    def forward(x_, l_, g_, w_):
        xn, mean, rstd = G.layer_norm(x_, g_, beta, eps)
        tw = _weights(l_, idx)
        xp = xn[src_of // k]
        yp = O.grouped_swiglu(xp, offsets, lambda e: w_[e], H, I, False)
        return O.combine(yp, row_of, tw, k), dict(mean=mean, rstd=rstd, tw=tw, xp=xp, yp=yp)

    loss = lambda *a: float((dy * forward(*a)[0]).sum())
    m = forward(x, logits, gamma, w)[1]
    dyp, dtw = G.combine_backward(dy, m["yp"], row_of, m["tw"], k)
    dl = G.route_backward(idx, m["tw"], dtw, E)
    ex = G.grouped_swiglu_backward(m["xp"], dyp, offsets, lambda e: w[e], H, I)
    dxn = G.permute_backward(ex["dx_perm"], row_of, k)
    dx, dgamma, _ = G.layer_norm_backward(dxn, x, gamma, m["mean"], m["rstd"])
    np.testing.assert_allclose(dl, differences(lambda v: loss(x, v, gamma, w), logits), atol=TOL)
    np.testing.assert_allclose(ex["dw"], differences(lambda v: loss(x, logits, gamma, v), w), atol=TOL)
    np.testing.assert_allclose(dgamma, differences(lambda v: loss(x, logits, v, w), gamma), atol=TOL)
    np.testing.assert_allclose(dx, differences(lambda v: loss(v, logits, gamma, w), x), atol=TOL)


PINS = dict(layer_norm=pin_layer_norm, combine=pin_combine, permute=pin_permute, route=pin_route,
            experts=pin_experts, whole_layer=pin_whole_layer)


@pytest.mark.parametrize("name", PINS)
def test_gradient_matches_differences(name):
    PINS[name]()


def _norm_without_projection(dy, x, gamma, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    a = dy * gamma
    return rstd[:, None] * (a - a.mean(1, keepdims=True)), (dy * xh).sum(0), dy.sum(0)


def _route_without_sum(idx, w, dw, E):
    dl = np.zeros((idx.shape[0], E))
    np.put_along_axis(dl, idx.astype(np.int64), w * dw, 1)
    return dl


def _ffn_with_plain_sigmoid(x, dy, wg, wu, wd):
    g, u = x @ wg.T, x @ wu.T
    s = 1 / (1 + np.exp(-g))
    dh = dy @ wd
    dg, du = dh * u * s, dh * g * s                      # silu' without its second term
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ (g * s * u), {}


@pytest.mark.parametrize("name,wrong", [
    ("layer_norm_backward", _norm_without_projection),
    ("route_backward", _route_without_sum),
    ("swiglu_ffn_backward", _ffn_with_plain_sigmoid),
    ("permute_backward", lambda d, row_of, k: d.reshape(-1, k, d.shape[1]).sum(1)),
    ("combine_backward", lambda dy, yp, row_of, w, k:
        (np.repeat(dy, k, 0) * w.reshape(-1, 1), (np.repeat(dy, k, 0) * yp).sum(1).reshape(w.shape))),
])
def test_planted_mistake_is_caught(monkeypatch, name, wrong):
    monkeypatch.setattr(G, name, wrong)
    failed = 0
    for pin in PINS.values():
        try:
            pin()
        except AssertionError:
            failed += 1
    assert failed >= 2
