"""A training step's operators around the products, in float64: normalization of rows with its
gradient, the gated activation with its gradient, and Newton-Schulz orthogonalization.

TEST INFRASTRUCTURE ONLY (see the package docstring).
"""

import numpy as np


def stats(h, eps, centred):
    """(hat, 1 / std) of rows."""
    h = np.asarray(h, np.float64)
    if centred:
        h = h - h.mean(axis=1, keepdims=True)
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + np.float64(np.float32(eps)))
    return h * r, r


def norm(h, gamma, eps, beta=None, centred=False):
    y = stats(h, eps, centred)[0] * np.asarray(gamma, np.float64)
    return y if beta is None else y + np.asarray(beta, np.float64)


def norm_bwd(dy, h, gamma, eps, centred=False, dres=None):
    """(dx, dgamma, dbeta)."""
    hat, r = stats(h, eps, centred)
    dy = np.asarray(dy, np.float64)
    dg = dy * np.asarray(gamma, np.float64)
    t = dg - hat * (dg * hat).mean(axis=1, keepdims=True)
    if centred:
        t = t - dg.mean(axis=1, keepdims=True)
    dx = r * t
    if dres is not None:
        dx = dx + np.asarray(dres, np.float64)
    return dx, (dy * hat).sum(axis=0), dy.sum(axis=0)


def sigmoid(g):
    t = np.exp(-np.abs(g))
    return np.where(g >= 0, 1.0, t) / (1.0 + t)


def swiglu(gu):
    gate, up = np.split(np.asarray(gu, np.float64), 2, axis=1)
    return gate * sigmoid(gate) * up


def swiglu_bwd(dy, gu):
    gate, up = np.split(np.asarray(gu, np.float64), 2, axis=1)
    dy, s = np.asarray(dy, np.float64), sigmoid(gate)
    return np.concatenate([dy * up * s * (1.0 + gate * sigmoid(-gate)), dy * gate * s], axis=1)


def orthogonalize(g, steps=5, coeffs=(3.4445, -4.7750, 2.0315), scale=1.0):
    """scale * X_steps: X_0 = g / |g| (Frobenius; a zero matrix stays zero), X <- a X + (b A + c A A) X with
    A = X X^T. For 3 dims one matrix each."""
    g = np.asarray(g, np.float64)
    if g.ndim == 3:
        return np.stack([orthogonalize(m, steps, coeffs, scale) for m in g])
    a, b, c = (np.float64(np.float32(v)) for v in coeffs)
    n = np.linalg.norm(g)
    x = g / n if n > 0 else g
    if x.shape[0] > x.shape[1]:
        x = x.T
    for _ in range(steps):
        A = x @ x.T
        x = a * x + (b * A + c * (A @ A)) @ x
    x = scale * x
    return x.T if g.shape[0] > g.shape[1] else x
