"""The gated operators on operands that the MFMA kernels do not take: many elements and few, columns
left over by whole eights, more blocks of rows than a grid has, sums that several of them share."""
import pytest

from test_gpu_gated import dgated_case, gated_case, i8_case
from test_gpu_gated_split import product, whole

pytestmark = pytest.mark.gpu


# (K or strides of no whole 16 bytes: every element on the generic kernels, on both sides of where they meet)
@pytest.mark.parametrize("shape", [(1031, 513, 71), (527, 1027, 33), (1024, 512, 20), (9, 700, 300), (8, 701, 1100), (33, 16, 515),
                                   (5, 17, 255), (4, 9, 257)])
@pytest.mark.parametrize("tB", [0, 1])
def test_any_k(gpu, shape, tB):
    for i, kind in enumerate(("bf16", "e4m3", "i8")):
        gated_case(gpu, i, *shape, tB, kind, ["bf16", "f32"][i % 2], "silu", "f32", pads=(1, 3, 5))
    dgated_case(gpu, 3, *shape, tB, "bf16", "f32", "gelu", pads=(3, 1, 1))
    dgated_case(gpu, 4, *shape, tB, "e4m3", "bf16", "relu", pads=(1, 0, 3))
    i8_case(gpu, 5, *shape, tB, "bf16", "gelu_tanh", "bf16", True, pads=(1, 5, 0))


@pytest.mark.parametrize("left", [1, 5, 7])
@pytest.mark.parametrize("rows", [1, 64, 777])
def test_left_columns(gpu, rows, left):
    N, K = 256 + left, 4112
    gated_case(gpu, left, rows, N, K, 1, "bf16", "bf16", "silu", "bf16")
    gated_case(gpu, left, rows, N, K, 1, "i8", "bf16", "silu", None, keep="")
    dgated_case(gpu, left, rows, N, K, 1, "bf16", "bf16", "silu")


@pytest.mark.parametrize("left", [1, 9, 15])
@pytest.mark.parametrize("rows", [1, 64, 777])
def test_left_columns_of_rows(gpu, rows, left):
    """B [K][N] with rows of whole 16 bytes and other columns; whole numbers."""
    import torch
    N, K = 256 + left, 1040
    for kind in ("bf16", "e4m3", "i8"):
        A = whole(rows, K, 2, 0, kind)
        Bg, Bu = (whole(K, N, 2, i, kind, 16 * i - left) for i in (1, 2))
        C, one = torch.empty(rows, N, device="cuda"), torch.ones(rows + N, device="cuda")
        g = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        if kind == "i8":
            gpu.run_gated_i8(A, one[:rows], Bg, one[:N], Bu, one[:N], C, act="relu", g=g)
        else:
            gpu.run_gated(A, Bg, Bu, C, act="relu", g=g)
        torch.cuda.synchronize()
        x, y = product(A, Bg, 0), product(A, Bu, 0)
        assert torch.equal(C, x.clamp(min=0) * y) and torch.equal(g, x.bfloat16()), kind
        if kind == "i8":
            gpu.run_i8(A, one[:rows], Bu, one[:N], C)
            torch.cuda.synchronize()
            assert torch.equal(C, y)


def test_more_blocks_of_rows_than_a_grid(gpu):
    """Whole numbers, exact sums: a workgroup takes several blocks of 4 rows."""
    import torch
    M, N, K = 270001, 11, 24
    A, Bg, Bu = whole(M, K, 2, 0, pad=1), whole(N, K, 2, 1, pad=1), whole(N, K, 2, 2, pad=3)
    C = torch.empty(M, N, device="cuda")
    gpu.run_gated(A, Bg, Bu, C, transB=1, act="relu")
    g, u = whole(M, N, 1, 3), whole(M, N, 1, 4)
    dg, du = torch.empty_like(C), torch.empty_like(C)
    sg, su = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    gpu.run_dgated(A, Bg, g, u, dg, du, transB=1, act="relu", dbias_g=sg, dbias_u=su)
    torch.cuda.synchronize()
    x, y = product(A, Bg, 1), product(A, Bu, 1)
    assert torch.equal(C, x.clamp(min=0) * y)
    on = (g > 0).float()
    wg, wu = x * u.float() * on, x * g.float() * on
    assert torch.equal(dg, wg) and torch.equal(du, wu)
    assert wg.abs().sum(0).max() < 2 ** 24 and wu.abs().sum(0).max() < 2 ** 24
    assert torch.equal(sg.double(), wg.double().sum(0)) and torch.equal(su.double(), wu.double().sum(0))


def test_the_same_bits(gpu):
    """Odd operands: sums in a fixed order, whatever the run."""
    import torch
    for M, N, K in ((2000, 5, 4097), (3, 1025, 4097), (1500, 700, 333)):
        A, B = whole(M, K, 100, 0).div(7), whole(N, K, 100, 1).div(7)
        g, u = whole(M, N, 100, 2).div(7), whole(M, N, 100, 3).div(7)
        out = []
        for _ in range(3):
            dg, du = torch.empty_like(g), torch.empty_like(g)
            s = torch.empty(2, N, device="cuda")
            gpu.run_dgated(A, B, g, u, dg, du, transB=1, act="silu", dbias_g=s[0], dbias_u=s[1])
            torch.cuda.synchronize()
            out.append((dg, du, s))
        assert all(torch.equal(a, b) for o in out[1:] for a, b in zip(o, out[0]))
