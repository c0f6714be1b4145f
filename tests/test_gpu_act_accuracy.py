"""The activations and their slopes into fp32 outputs, over the whole of their argument: products
whose value is exact, so that nothing but the activation's own error is left.

Bounds, u = 2^-24.  The hardware's exponential and reciprocal are good to 2 u each, an exponent's
rounding moves the exponential by itself times that.  GELU (erf): q = 1 - Phi(|z|) is fitted to
7e-8 (1 + 2 z^2) of itself, and its exponent (three roundings), seven coefficients, t and two
products add u (1.5 z^2 + 14).  The logistic of v = k z (k roundings of v): (1 - s) (2 k u |v| / 2 +
2 u) + 3 u of itself.  Results under 1e-36 may be flushed.
"""
import numpy as np
import pytest
from scipy.special import erfc

from oracle import mlp

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
N = 4096
TINY = 1e-36


def arguments(rng):
    z = np.concatenate([np.linspace(-14, 14, 2048), rng.uniform(-1, 1, 1024), rng.uniform(-6, 0, 512),
                        np.ldexp(rng.choice([-1.0, 1.0], 496) * rng.uniform(1, 2, 496), rng.integers(-60, 60, 496)),
                        [0.0, 1e-30, -1e-30, 100.0, -100.0, 3e4, -3e4, 1e20, -1e20, 3e38, -3e38, 13.2, -13.2, 64.0, -64.0, 1.0]])
    return z.astype(np.float32)


def act(z, kind):
    """mlp.act, with GELU's tanh form by the logistic: in 64 bits 1 + tanh(u) is 0 from u = -19 on,
    where z logistic(2u) is 1e-16."""
    return z * mlp._logistic(2 * mlp.C0 * (z + mlp.C1 * z ** 3)) if kind == "gelu_tanh" else mlp.act(z, kind)


def bounds(z, kind):
    """Of act(z) and of its slope."""
    a = np.abs(z)
    value, slope = np.abs(act(z, kind)), np.abs(mlp.slope(z, kind))
    if kind in ("none", "relu"):
        return 0 * z, 0 * z
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        if kind == "gelu":
            rel = 7e-8 * (1 + 2 * z * z) + U * (1.5 * z * z + 14)
            q, phi = 0.5 * erfc(a / np.sqrt(2.0)), np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
            dq = np.where(q > 0, q * np.minimum(rel, 1e300), 0)
            return (a * dq + 2 * U * value + 2 * U * np.where(z > 0, a, 0) + TINY,
                    dq + np.where(phi > 0, a * phi * U * (1.5 * z * z + 6), 0) + 3 * U * np.maximum(slope, z > 0) + TINY)
        if kind == "silu":
            v, k, inner = a, 2, np.ones_like(z)
        else:
            v = np.minimum(2 * mlp.C0 * (a + mlp.C1 * a ** 3), 1e4)
            c = np.minimum(a, 64.0)
            k, inner = 5, 2 * mlp.C0 * (1 + 3 * mlp.C1 * c * c)
        s = mlp._logistic(np.sign(z) * v)
        ds = s * ((1 - s) * (2 * k * U * v + 2 * U) + 3 * U)
        c = np.minimum(a, 1e4)
        return (a * ds + 2 * U * value + TINY * np.maximum(a, 1),
                ds * (1 + 2 * c * inner) + 6 * U * (1 + c * s * (1 - s) * inner) + TINY * (1 + c * inner))


def check(got, want, bound, what, z):
    bad = ~(np.abs(got - want) <= bound)
    i = np.argmax(np.where(bound > 0, np.abs(got - want) / np.maximum(bound, 1e-300), bad))
    assert not bad.any(), f"{what}: {bad.sum()} outside, worst at z = {z.flat[i]}: {got.flat[i]} for {want.flat[i]}, bound {bound.flat[i]}"


@pytest.mark.parametrize("kind", mlp.ACTS)
@pytest.mark.parametrize("M", [1, 130])
def test_values(gpu, kind, M):
    """A zero product and the argument as bias."""
    import torch
    z = arguments(np.random.default_rng(M))
    assert z.size == N
    A, B = torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, 8, dtype=torch.bfloat16, device="cuda")
    C = torch.full((M, N), float("nan"), device="cuda")
    gpu.run_act(A, B, C, transB=1, act=kind, bias=torch.from_numpy(z).cuda())
    torch.cuda.synchronize()
    zv = z.astype(np.float64)
    got = C.double().cpu().numpy()
    assert (got == got[:1]).all()
    check(got[0], act(zv, kind), bounds(zv, kind)[0], kind, zv)


@pytest.mark.parametrize("kind", mlp.ACTS)
@pytest.mark.parametrize("M", [3, 130])
def test_slopes(gpu, kind, M):
    """A product of ones."""
    import torch
    rng = np.random.default_rng(10 + M)
    z = torch.from_numpy(np.stack([arguments(rng) for _ in range(M)])).to(torch.bfloat16).cuda()
    A, B = torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda"), torch.zeros(N, 8, dtype=torch.bfloat16, device="cuda")
    A[:, 0] = B[:, 0] = 1
    C = torch.full((M, N), float("nan"), device="cuda")
    gpu.run_dact(A, B, C, z, transB=1, act=kind)
    torch.cuda.synchronize()
    zv = z.double().cpu().numpy()
    # (3e38 is 2^128 - 2^119 at most in bf16: finite)
    assert np.isfinite(zv).all()
    with np.errstate(over="ignore", invalid="ignore"):
        want = mlp.slope(np.clip(zv, -1e4, 1e4), kind)
    check(C.double().cpu().numpy(), want, bounds(np.clip(zv, -1e4, 1e4), kind)[1], kind + "'", zv)
