"""Layer norm's mean on the GPU: rows whose mean is large against their spread, down to constant
rows, in every kernel (by width and rows).

Bounds.  u = 2^-24.  An fp32 row's sum is taken in 64 bits, so its mean is the fp32 number next to the true
one, m, and what that rounding leaves, at most u |mean|, is taken out again: m and the deviations
x - m of a constant row are exact.  So are they for bf16 rows, whose sums fp32 holds.  The squares' sum is fp32, d the longest run of its additions.
"""
import numpy as np
import pytest

from oracle import mlp

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SHAPES = [(6, 5), (6, 200), (300, 200), (6, 4099), (300, 1100), (300, 5120), (6, 12000), (6, 20480), (6, 40001)]


def chain(N):
    """A lane takes 1/64 of the row (a 256th past 32768 columns), then a tree."""
    return -(-N // 64) + 16


def run(gpu, x, eps, gamma=None, beta=None):
    import torch
    y = torch.full(x.shape, float("nan"), device="cuda")  # fp32
    mean, rstd = (torch.full((x.shape[0],), float("nan"), device="cuda") for _ in range(2))
    gpu.layernorm(x, y, gamma=gamma, beta=beta, eps=eps, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    return tuple(t.cpu().numpy().astype(np.float64) for t in (y, mean, rstd))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_constant_rows(gpu, shape, kind):
    import torch
    M, N = shape
    c32 = torch.from_numpy(np.resize(np.array([0.1, 3.3, 1.7, 1000.1, 1e6 + 0.3, -77777.7], dtype=np.float32), M))
    c = c32.to(torch.bfloat16 if kind == "bf16" else torch.float32)
    x, c = c[:, None].repeat(1, N).cuda(), c.double().numpy()[:, None]
    rng = np.random.default_rng(N)
    g, b = (rng.standard_normal(N).astype(np.float32) for _ in range(2))
    eps = 1e-5
    y, mean, rstd = run(gpu, x, eps, torch.from_numpy(g).cuda(), torch.from_numpy(b).cuda())
    assert np.array_equal(y, np.broadcast_to(b.astype(np.float64), y.shape)), np.abs(y - b).max()
    assert np.array_equal(mean, c[:, 0]), mean - c[:, 0]
    assert (np.abs(rstd * np.sqrt(eps) - 1) <= 4 * U).all(), rstd


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("at", [1e4, -1e6])
def test_rows_far_from_zero(gpu, shape, at):
    import torch
    M, N = shape
    rng = np.random.default_rng(N + M)
    x32 = (at + rng.standard_normal((M, N))).astype(np.float32)
    xv = x32.astype(np.float64)
    y, mean, rstd = run(gpu, torch.from_numpy(x32).cuda(), 1e-3)
    want, mu, r = mlp.layernorm(xv, eps=1e-3)
    d = chain(N)
    e = U * np.abs(mu)  # |mu - m|
    v = np.abs(xv - mu[:, None])
    # the deviations' mean square about m, less e^2
    e_r = r * (0.5 * r * r * (d + 6) * U * ((v * v).mean(1) + e * e) + 4 * U)
    assert (np.abs(mean - mu) <= e * 1.001).all(), np.abs(mean - mu).max()
    assert (np.abs(rstd - r) <= e_r).all(), np.abs(rstd - r).max()
    bound = (v + e[:, None]) * (4 * U * r + e_r)[:, None] + 2 * U * np.abs(want)
    assert (np.abs(y - want) <= bound).all(), (np.abs(y - want) / bound).max()


@pytest.mark.parametrize("shape", SHAPES)
def test_infinite_rows(gpu, shape):
    """An infinity gives its row that mean and no numbers; the others keep theirs."""
    import torch
    M, N = shape
    x = torch.randn(M, N, device="cuda")
    x[1, 0], x[3, N - 1], x[4, N // 2] = float("inf"), float("-inf"), float("nan")
    y, mean, rstd = run(gpu, x, 1e-5)
    assert mean[1] == np.inf and mean[3] == -np.inf and np.isnan(mean[4])
    assert np.isnan(y[[1, 3, 4]]).all() and np.isnan(rstd[[1, 3, 4]]).all()
    rest = [i for i in range(M) if i not in (1, 3, 4)]
    assert np.isfinite(y[rest]).all() and np.isfinite(mean[rest]).all() and np.isfinite(rstd[rest]).all()


@pytest.mark.parametrize("shape", [(3, 0), (0, 7)])
def test_nothing_to_normalise(gpu, shape):
    import torch
    x = torch.empty(shape, device="cuda")
    mean, rstd = torch.full((shape[0],), 5.0, device="cuda"), torch.full((shape[0],), 6.0, device="cuda")
    gpu.layernorm(x, torch.empty_like(x), mean=mean, rstd=rstd)
    if shape[0]:
        gpu.layernorm_grad(x, x, mean, rstd, torch.empty_like(x), dgamma=torch.empty(0, device="cuda"),
                           dbeta=torch.empty(0, device="cuda"))
    torch.cuda.synchronize()
    assert (mean == 5).all() and (rstd == 6).all()
