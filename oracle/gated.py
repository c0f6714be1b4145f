"""The gated feed-forward operators in float64 (numpy), from their definitions: both projections
with the gate, the product that runs back through it, rows as 8-bit integers and their products.
Test infrastructure only; shares nothing with the library.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

from . import mlp


def run_gated(A, Bg, Bu, alpha, kind, bias_g=None, bias_u=None, transB=0):
    """(H, G, U, Sg, Su): S the sums of the magnitudes of the products' terms."""
    G, Sg = mlp.product(A, Bg, alpha, 0, transB)
    U, Su = mlp.product(A, Bu, alpha, 0, transB)
    if bias_g is not None:
        G = G + bias_g
    if bias_u is not None:
        U = U + bias_u
    return mlp.act(G, kind) * U, G, U, Sg, Su


def run_dgated(A, B, alpha, kind, g, u, transB=0):
    """(dG, dU, H, P, S) with P the product before the gate."""
    P, S = mlp.product(A, B, alpha, 0, transB)
    a = mlp.act(g, kind)
    return P * u * mlp.slope(g, kind), P * a, a * u, P, S


def quantize_i8(x):
    """Rows of finite values -> (codes, exact scales in float64).  The quotient decided in rationals."""
    x = np.asarray(x, dtype=np.float64)
    q = np.zeros(x.shape, dtype=np.int8)
    top = np.abs(x).max(1) if x.shape[1] else np.zeros(x.shape[0])
    for r in range(x.shape[0]):
        if top[r] > 0:
            t = Fraction(float(top[r]))
            # (round() of a Fraction: to the nearest whole number, ties to even)
            q[r] = [round(Fraction(float(v)) * 127 / t) for v in x[r]]
    return q, top / 127.0


def product_i8(A, sa, B, sb, transB=0):
    """The scaled product and its exact sums of whole numbers."""
    b = B.astype(np.int64)
    sums = A.astype(np.int64) @ (b.T if transB else b)
    return sums * np.asarray(sa, np.float64)[:, None] * np.asarray(sb, np.float64), sums
