"""The MLP-block operators in float64 (numpy), from their definitions: products with a bias,
an activation and a residual, the product that runs back through the activation, layer norm
and its gradient.  Test infrastructure only; shares nothing with the library.

Each product also returns what its error bounds are made of: S = |alpha| * sum |a b|.
"""
from __future__ import annotations

import numpy as np
from scipy.special import erfc

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
C0, C1 = np.sqrt(2.0 / np.pi), 0.044715


def _logistic(z):
    with np.errstate(over="ignore"):
        return np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))


def act(z, kind):
    z = np.asarray(z, dtype=np.float64)
    if kind == "none":
        return z
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "gelu":
        return z * 0.5 * erfc(-z / np.sqrt(2.0))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(C0 * (z + C1 * z ** 3)))
    if kind == "silu":
        return z * _logistic(z)
    raise ValueError(kind)


def slope(z, kind):
    """d act / dz (0 at z = 0 for relu)."""
    z = np.asarray(z, dtype=np.float64)
    if kind == "none":
        return np.ones_like(z)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu":
        return 0.5 * erfc(-z / np.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    if kind == "gelu_tanh":
        t = np.tanh(C0 * (z + C1 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * C0 * (1.0 + 3.0 * C1 * z * z)
    if kind == "silu":
        s = _logistic(z)
        return s * (1.0 + z * (1.0 - s))
    raise ValueError(kind)


def product(A, B, alpha, transA=0, transB=0):
    """alpha * op(A) op(B) and the sum of the magnitudes of its terms."""
    a = A.T if transA else A
    b = B.T if transB else B
    return alpha * (a @ b), abs(alpha) * (np.abs(a) @ np.abs(b))


def run_act(A, B, alpha, kind, bias=None, residual=None, beta=1.0, transA=0, transB=0):
    """(C, Z, S)."""
    Z, S = product(A, B, alpha, transA, transB)
    if bias is not None:
        Z = Z + bias
    C = act(Z, kind)
    if residual is not None and beta != 0.0:
        C = C + beta * residual
    return C, Z, S


def run_dact(A, B, alpha, kind, z, transA=0, transB=0):
    """(D, column sums of D, P, S) with P the product before the slope."""
    P, S = product(A, B, alpha, transA, transB)
    D = P * slope(z, kind)
    return D, D.sum(0), P, S


def from_mx(values, scales):
    """Values of block-scaled codes: `values` the decoded E4M3 elements, one scale byte per 32."""
    f = np.ldexp(1.0, scales.astype(np.int64) - 127)
    return values * np.repeat(f, 32, axis=1)[:, :values.shape[1]]


def layernorm(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd)."""
    mu = x.mean(1)
    d = x - mu[:, None]
    r = 1.0 / np.sqrt((d * d).mean(1) + eps)
    y = d * r[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mu, r


def layernorm_grad(dy, x, mean, rstd, gamma=None, residual=None):
    """(dx, dgamma, dbeta)."""
    n = (x - mean[:, None]) * rstd[:, None]
    g = dy if gamma is None else dy * gamma
    dx = rstd[:, None] * (g - g.mean(1)[:, None] - n * (g * n).mean(1)[:, None])
    if residual is not None:
        dx = dx + residual
    return dx, (dy * n).sum(0), dy.sum(0)
