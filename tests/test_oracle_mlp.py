"""Pins of the MLP-block oracle: hand values, torch's own functions as library routines, and
every gradient against differences."""
import numpy as np
import pytest

from oracle import mlp


def test_hand_values():
    z = np.array([-2.0, 0.0, 2.0])
    assert np.array_equal(mlp.act(z, "relu"), [0.0, 0.0, 2.0])
    assert np.array_equal(mlp.slope(z, "relu"), [0.0, 0.0, 1.0])
    assert np.allclose(mlp.act(z, "silu"), [-2 / (1 + np.e ** 2), 0, 2 / (1 + np.e ** -2)], rtol=1e-15)
    # Phi(2) = 0.97724986805182079
    assert np.allclose(mlp.act(z, "gelu"), [-2 * (1 - 0.97724986805182079), 0, 2 * 0.97724986805182079], rtol=1e-13)
    x = np.array([[1.0, 2.0, 3.0, 6.0]])  # mean 3, variance 3.5
    y, mu, r = mlp.layernorm(x, np.array([1.0, 1.0, 2.0, 1.0]), np.array([0.0, 0.5, 0.0, 0.0]), eps=0.5)
    assert mu[0] == 3.0 and r[0] == 0.5
    assert np.array_equal(y, [[-1.0, 0.0, 0.0, 1.5]])


@pytest.mark.parametrize("kind", mlp.ACTS)
def test_activations_against_torch(kind):
    torch = pytest.importorskip("torch")
    f = {"none": lambda t: t, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
         "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[kind]
    z = np.linspace(-12.0, 12.0, 997)
    t = torch.from_numpy(z).requires_grad_(True)
    out = f(t)
    (g,) = torch.autograd.grad(out.sum(), t)
    assert np.allclose(mlp.act(z, kind), out.detach().numpy(), rtol=1e-9, atol=1e-14)
    assert np.allclose(mlp.slope(z, kind), g.numpy(), rtol=1e-9, atol=1e-13)


@pytest.mark.parametrize("kind", mlp.ACTS)
def test_slope_is_the_difference_quotient(kind):
    z = np.linspace(-6.0, 6.0, 301) + 1e-3  # off the kink of relu
    h = 1e-5
    d = (mlp.act(z + h, kind) - mlp.act(z - h, kind)) / (2 * h)
    # central differences: h^2 |act'''| / 6 (|act'''| < 4) plus rounding 2^-53 |act| / h
    assert np.abs(d - mlp.slope(z, kind)).max() <= 4 * h * h / 6 + 2.0 ** -52 * 6 / h


def test_products_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(0)
    A, B, bias = rng.standard_normal((4, 6)), rng.standard_normal((6, 5)), rng.standard_normal(5)
    W2, dY = rng.standard_normal((5, 3)), rng.standard_normal((4, 3))
    loss = lambda b: float(((mlp.run_act(A, B, 0.5, "gelu", bias=b)[0] @ W2) * dY).sum())  # noqa: E731
    z = mlp.run_act(A, B, 0.5, "gelu", bias=bias)[1]
    D, db, _, _ = mlp.run_dact(dY, W2, 1.0, "gelu", z, transB=1)
    h = 1e-6
    for n in range(5):
        e = np.eye(5)[n] * h
        assert abs((loss(bias + e) - loss(bias - e)) / (2 * h) - db[n]) <= 1e-7
    assert np.allclose(D.sum(0), db)


@pytest.mark.parametrize("n", [1, 7, 33])
def test_layernorm_grad_is_the_difference_quotient(n):
    rng = np.random.default_rng(n)
    x, dy, res = (rng.standard_normal((3, n)) for _ in range(3))
    g, b = rng.standard_normal(n), rng.standard_normal(n)
    loss = lambda x, g, b: float((mlp.layernorm(x, g, b, eps=0.1)[0] * dy).sum())  # noqa: E731
    _, mu, r = mlp.layernorm(x, g, b, eps=0.1)
    dx, dg, db = mlp.layernorm_grad(dy, x, mu, r, g)
    assert np.array_equal(mlp.layernorm_grad(dy, x, mu, r, g, residual=res)[0], dx + res)
    h = 1e-6
    for i in range(n):
        e = np.eye(n)[i] * h
        assert abs((loss(x, g + e, b) - loss(x, g - e, b)) / (2 * h) - dg[i]) <= 1e-7
        assert abs((loss(x, g, b + e) - loss(x, g, b - e)) / (2 * h) - db[i]) <= 1e-7
        for m in range(3):
            d = np.zeros_like(x)
            d[m, i] = h
            assert abs((loss(x + d, g, b) - loss(x - d, g, b)) / (2 * h) - dx[m, i]) <= 1e-6


def test_from_mx_spreads_the_scales():
    v = np.ones((1, 40))
    assert np.array_equal(mlp.from_mx(v, np.array([[128, 126]], dtype=np.uint8)), [[2.0] * 32 + [0.5] * 8])
