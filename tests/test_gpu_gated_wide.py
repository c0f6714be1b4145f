"""The gated operators on more columns than the generic kernels take in one launch: 2^26 to a launch, where
2^27 columns for few elements would be 2^32 threads, and with column sums 2^22 where a partial row of them
does not fit the workspace.  Whole numbers, exact sums."""
import pytest

from test_gpu_gated_split import whole

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(1, (1 << 27) + 11, 1), (3, (1 << 26) + 1, 2)])
@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_columns_past_a_launch(gpu, shape, kind):
    import torch
    M, N, K = shape
    A, Bg, Bu = whole(M, K, 5, 0, kind), whole(K, N, 5, 1, kind), whole(K, N, 5, 2, kind)
    C = torch.full((M, N), -7.0, dtype=torch.bfloat16, device="cuda")
    if kind == "i8":
        one = torch.ones(N, device="cuda")
        gpu.run_gated_i8(A, one[:M], Bg, one, Bu, one, C, act="relu")
    else:
        gpu.run_gated(A, Bg, Bu, C, act="relu")
    torch.cuda.synchronize()
    for m in range(M):
        x, y = (sum(A[m, k].float() * B[k].float() for k in range(K)) for B in (Bg, Bu))
        assert torch.equal(C[m], (x.clamp(min=0) * y).bfloat16())
    if kind == "i8":
        R = C.clone()
        gpu.run_i8(A, one[:M], Bu, one, C, residual=R)
        torch.cuda.synchronize()
        for m in range(M):
            y = sum(A[m, k].float() * Bu[k].float() for k in range(K))
            assert torch.equal(C[m], (y + R[m].float()).bfloat16())
    else:
        g, u = (Bg, Bu) if M == K == 1 else (C, C.clone())
        dg, du = torch.empty_like(C), torch.empty_like(C)
        gpu.run_dgated(A, Bu, g, u, dg, du, act="relu")
        torch.cuda.synchronize()
        for m in range(M):
            p, on = sum(A[m, k].float() * Bu[k].float() for k in range(K)), (g[m] > 0).float()
            assert torch.equal(dg[m], (p * u[m].float() * on).bfloat16())
            assert torch.equal(du[m], (p * g[m].float() * on).bfloat16())


# few elements and many, K that the MFMA kernels take (B [N][K]) and not
@pytest.mark.parametrize("shape", [(3, (1 << 23) + 13, 3), (70, (1 << 23) + 9, 3), (70, (1 << 23) + 16, 8)])
@pytest.mark.parametrize("tB", [0, 1])
@pytest.mark.parametrize("sums", ["gu", "u"])
def test_sums_of_more_columns_than_the_workspace_holds(gpu, shape, tB, sums):
    import torch
    M, N, K = shape
    A, B = whole(M, K, 2, 0), whole(*((N, K) if tB else (K, N)), 2, 1)
    g, u = whole(M, N, 2, 2), whole(M, N, 2, 3)
    dg, du = torch.empty_like(g), torch.empty_like(g)
    sg, su = (torch.full((N,), -7.0, device="cuda") for _ in range(2))
    gpu.run_dgated(A, B, g, u, dg, du, transB=tB, act="relu", dbias_g=sg if "g" in sums else None, dbias_u=su)
    torch.cuda.synchronize()
    wg, wu = torch.zeros(N, device="cuda"), torch.zeros(N, device="cuda")
    for m in range(M):
        p = sum(A[m, k].float() * (B[:, k] if tB else B[k]).float() for k in range(K))
        x, y = p * u[m].float() * (g[m] > 0).float(), p * g[m].float().clamp(min=0)
        assert torch.equal(dg[m], x.bfloat16()) and torch.equal(du[m], y.bfloat16()), m
        wg += x
        wu += y
    assert torch.equal(su, wu)
    assert torch.equal(sg, wg) if "g" in sums else (sg == -7).all()
