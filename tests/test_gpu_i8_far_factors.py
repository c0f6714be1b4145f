"""8-bit integer products whose factors are far apart: sum * scale_a * scale_b lies in fp32's range
where sum * scale_a alone does not (a row that held bf16's lowest value has a factor of 2.7e36), and
where one of the factors is subnormal.

Bounds: the sum's conversion and two products, U = 2^-24 each, so (1 + U)^3 - 1 < 4 U of the exact
product, and 2^-149 where that is subnormal; a gated one has seven roundings, under 8 U."""
import numpy as np
import pytest

from oracle import gated
from test_gpu_gated import U, host, matrix

pytestmark = pytest.mark.gpu

# few rows, tiles, split tiles, operands of the generic kernels (few elements and many)
SHAPES = [(5, 64, 272), (40, 136, 8192), (100, 304, 128), (300, 512, 96), (513, 1040, 272), (3, 17, 5), (65, 129, 71),
          (900, 700, 33), (70, 83, 96)]


def factors(rng, n, low, high):
    import torch
    v = np.ldexp(rng.uniform(1, 2, n), rng.integers(low, high + 1, n)).astype(np.float32)
    return torch.from_numpy(v).cuda(), v.astype(np.float64)


def near(got, want, bound, what):
    off = np.abs(got - want)
    assert np.isfinite(got).all(), what
    assert (off <= bound).all(), (what, (off / bound).max())


# (exponents of scale_a and scale_b; results between 2^-149 and 2^128 throughout)
FAR = [(100, 120, -119, -90), (-119, -90, 100, 120), (60, 70, -70, -60), (-149, -140, 100, 120), (100, 120, -149, -140)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("tB", [0, 1])
@pytest.mark.parametrize("far", FAR)
def test_products(gpu, shape, tB, far):
    import torch
    M, N, K = shape
    rng = np.random.default_rng(5)
    A, Av = matrix(rng, M, K, "i8")
    B, Bv = matrix(rng, *((N, K) if tB else (K, N)), "i8")
    (sa, sav), (sb, sbv) = factors(rng, M, *far[:2]), factors(rng, N, *far[2:])
    C = torch.empty(M, N, device="cuda")
    gpu.run_i8(A, sa, B, sb, C, transB=tB)
    torch.cuda.synchronize()
    P = gated.product_i8(Av, sav, Bv, sbv, tB)[0]
    assert np.abs(P).max() < 2.0 ** 127
    near(host(C), P, 4 * U * np.abs(P) + 2.0 ** -149, (shape, tB, far))


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("tB", [0, 1])
def test_gated_products(gpu, shape, tB):
    """A gate near 1 whose factors are far apart, times a factor of the same row."""
    import torch
    M, N, K = shape
    rng = np.random.default_rng(6)
    A, Av = matrix(rng, M, K, "i8")
    (Bg, Bgv), (Bu, Buv) = (matrix(rng, *((N, K) if tB else (K, N)), "i8") for _ in range(2))
    (sa, sav), (sg, sgv), (su, suv) = factors(rng, M, 100, 115), factors(rng, N, -125, -115), factors(rng, N, -110, -100)
    C = torch.empty(M, N, device="cuda")
    gpu.run_gated_i8(A, sa, Bg, sg, Bu, su, C, transB=tB, act="relu")
    torch.cuda.synchronize()
    G, V = gated.product_i8(Av, sav, Bgv, sgv, tB)[0], gated.product_i8(Av, sav, Buv, suv, tB)[0]
    H = np.maximum(G, 0) * V
    near(host(C), H, 8 * U * np.abs(H) + 2.0 ** -149, (shape, tB))


def test_the_lowest_value_in_a_row(gpu):
    """Quantised with bf16's lowest value among its elements, times weights, and a bias; its neighbours keep
    the bits that they have beside an ordinary row (the bias's rounding is one more)."""
    import torch
    for M, N, K in ((5, 64, 272), (300, 512, 96), (65, 129, 71)):
        r = torch.Generator().manual_seed(M)
        x = torch.randn(M, K, generator=r).bfloat16()
        w, bias = torch.randn(N, K, generator=r) * 1e-3, torch.randn(N, generator=r)
        low = x.clone()
        low[1, 3] = torch.finfo(torch.bfloat16).min
        out = []
        for v in (x, low):
            q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
            b, sb = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
            gpu.quantize_i8(v.cuda(), q, s)
            gpu.quantize_i8(w.cuda(), b, sb)
            C = torch.empty(M, N, device="cuda")
            gpu.run_i8(q, s, b, sb, C, transB=1, bias=bias.cuda())
            torch.cuda.synchronize()
            P = gated.product_i8(q.cpu().numpy(), s.cpu().numpy(), b.cpu().numpy(), sb.cpu().numpy(), 1)[0]
            near(host(C), P + bias.numpy(), 4 * U * np.abs(P) + U * np.abs(P + bias.numpy()) + 2.0 ** -149, (M, N, K))
            out.append(C)
        rest = [i for i in range(M) if i != 1]
        assert torch.equal(out[0][rest], out[1][rest])
