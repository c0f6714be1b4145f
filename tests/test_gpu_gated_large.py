"""The gated operators on outputs and operands past the limits of one launch: rows in blocks, because
32-bit offsets into A or the workspace's partial sums end.  Whole numbers, so that every sum is exact
in whatever order."""
import pytest

pytestmark = pytest.mark.gpu


def whole(rows, cols, span, seed):
    import torch
    r = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(-span, span + 1, (rows, cols), generator=r, device="cuda").to(torch.bfloat16)


def test_rows_past_the_offsets_into_A():
    """A of 2.6 GB at a stride of 4096: two blocks of rows."""
    import torch
    import dense_blas3_gemm_amd as d
    M, N, K = 320000, 72, 16
    buf = torch.empty(M, 4096, dtype=torch.bfloat16, device="cuda")
    A = buf[:, :K]
    A.copy_(whole(M, K, 2, 0))
    Bg, Bu = whole(N, K, 2, 1), whole(N, K, 2, 2)
    C = torch.empty(M, N, device="cuda")
    h = d.Gemm(0)
    try:
        h.run_gated(A, Bg, Bu, C, transB=1, act="relu")
        x = A.float()
        want = (x @ Bg.float().t()).clamp(min=0) * (x @ Bu.float().t())
        torch.cuda.synchronize()
        assert torch.equal(C, want)
        A8, ones = torch.empty(M, 8192, dtype=torch.int8, device="cuda")[:, :K], torch.ones(M, device="cuda")
        A8.copy_(A)
        h.run_i8(A8, ones, Bg.to(torch.int8), ones[:N], C, transB=1)
        torch.cuda.synchronize()
        assert torch.equal(C, x @ Bg.float().t())
    finally:
        h.close()


def test_sums_past_the_workspace():
    """One row of partial sums to 64 rows: 100100 x 8200 would need 205 MB of it; and the last columns
    past a whole eight."""
    import torch
    import dense_blas3_gemm_amd as d
    M, N, K = 100100, 8203, 16
    A, B = whole(M, K, 1, 0), whole(N, K, 1, 1)
    g, u = whole(M, N, 1, 2), whole(M, N, 2, 3)
    dg, du = torch.empty_like(g), torch.empty_like(u)
    sg, su = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    h = d.Gemm(0)
    try:
        h.run_dgated(A, B, g, u, dg, du, transB=1, act="relu", dbias_g=sg, dbias_u=su)
        torch.cuda.synchronize()
        wg, wu = torch.zeros(N, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
        for m in range(0, M, 10010):
            s = slice(m, m + 10010)
            p = A[s].float() @ B.float().t()
            x, y = p * u[s] * (g[s] > 0), p * g[s].clamp(min=0)
            assert torch.equal(dg[s].float(), x) and torch.equal(du[s].float(), y), m
            wg += x.double().sum(0)
            wu += y.double().sum(0)
        # (sums under 2^24)
        assert torch.equal(sg.double(), wg) and torch.equal(su.double(), wu)
    finally:
        h.close()
        del g, u, dg, du
        torch.cuda.empty_cache()
