"""Pins of the gated operators' oracle: hand values, and the gradient against differences."""
import numpy as np
import pytest

from oracle import gated, mlp


def test_hand_values():
    A, Bg, Bu = np.array([[1.0, 2.0]]), np.array([[3.0, -1.0], [1.0, -1.0]]), np.array([[1.0, 5.0], [0.5, 1.0]])
    H, G, U, Sg, Su = gated.run_gated(A, Bg, Bu, 2.0, "relu", bias_g=np.array([1.0, 1.0]), bias_u=np.array([0.0, 2.0]))
    assert np.array_equal(G, [[11.0, -5.0]]) and np.array_equal(U, [[4.0, 16.0]])
    assert np.array_equal(H, [[44.0, 0.0]]) and np.array_equal(Sg, [[10.0, 6.0]]) and np.array_equal(Su, [[4.0, 14.0]])
    assert np.array_equal(gated.run_gated(A, Bg.T, Bu.T, 2.0, "relu", transB=1)[0],
                          gated.run_gated(A, Bg, Bu, 2.0, "relu")[0])


def test_codes_by_hand():
    # 63.5 lies between 63 and 64: to the even one; -2.5 steps of a row whose step is 1
    q, s = gated.quantize_i8(np.array([[127.0, 63.5, -2.5, 0.4], [2.0, 1.0, -1.0, 0.0], [0.0, 0.0, 0.0, 0.0]]))
    assert np.array_equal(q, [[127, 64, -2, 0], [127, 64, -64, 0], [0, 0, 0, 0]])
    assert np.array_equal(s, [1.0, 2.0 / 127.0, 0.0])
    P, sums = gated.product_i8(q[:1], s[:1], np.array([[1], [2], [-1], [5]], np.int8), np.array([0.5]))
    assert sums[0, 0] == 127 + 128 + 2 and P[0, 0] == 128.5


def test_codes_stand_for_values_within_half_a_step():
    rng = np.random.default_rng(0)
    x = np.ldexp(rng.standard_normal((7, 65)), rng.integers(-20, 20, (7, 1)))
    q, s = gated.quantize_i8(x)
    assert (np.abs(q * s[:, None] - x) <= s[:, None] * (0.5 + 1e-12)).all()
    assert (np.abs(q.astype(int)).max(1) == 127).all()


@pytest.mark.parametrize("kind", mlp.ACTS)
def test_gradient_is_the_difference_quotient(kind):
    """Of a whole block's loss, in both projections' weights and biases."""
    rng = np.random.default_rng(1)
    X, Wg, Wu, Wd = (rng.standard_normal(s) for s in ((4, 6), (6, 5), (6, 5), (5, 3)))
    bg, bu, dY = rng.standard_normal(5), rng.standard_normal(5), rng.standard_normal((4, 3))
    loss = lambda Wg, Wu, bg, bu: float(((gated.run_gated(X, Wg, Wu, 0.5, kind, bg, bu)[0] @ Wd) * dY).sum())  # noqa: E731
    _, G, U, _, _ = gated.run_gated(X, Wg, Wu, 0.5, kind, bg, bu)
    dG, dU, H, P, _ = gated.run_dgated(dY, Wd, 1.0, kind, G, U, transB=1)
    assert np.array_equal(H, mlp.act(G, kind) * U) and np.allclose(P, dY @ Wd.T)
    h = 1e-6
    for n in range(5):
        e = np.eye(5)[n] * h
        assert abs((loss(Wg, Wu, bg + e, bu) - loss(Wg, Wu, bg - e, bu)) / (2 * h) - dG.sum(0)[n]) <= 1e-6
        assert abs((loss(Wg, Wu, bg, bu + e) - loss(Wg, Wu, bg, bu - e)) / (2 * h) - dU.sum(0)[n]) <= 1e-6
    dWg, dWu = 0.5 * X.T @ dG, 0.5 * X.T @ dU
    for i, j in ((0, 0), (3, 2), (5, 4)):
        E = np.zeros((6, 5))
        E[i, j] = h
        assert abs((loss(Wg + E, Wu, bg, bu) - loss(Wg - E, Wu, bg, bu)) / (2 * h) - dWg[i, j]) <= 1e-6
        assert abs((loss(Wg, Wu + E, bg, bu) - loss(Wg, Wu - E, bg, bu)) / (2 * h) - dWu[i, j]) <= 1e-6
