"""The gated operators on more columns than the generic kernels take in one launch: 2^26 to a launch, where
2^27 columns for few elements would be 2^32 threads.  Whole numbers, exact sums."""
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
