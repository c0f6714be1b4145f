"""The gated and 8-bit integer operators on every kernel that they are dispatched to (tests/gated_plan.py, whose
shapes are held to that by tests/test_gated_plans.py): few rows at each width, tiles of each size, split and
whole, products in two launches along either side.  Whole numbers with every sum under 2^24, so that any order
of additions gives the exact sum, and what follows it is compared bit by bit."""
import pytest

from gated_plan import FORMS, PAD, SHAPES, plan
from test_gpu_gated_split import product, whole

pytestmark = pytest.mark.gpu


def out(M, N, pad, dt):
    """(the matrix, its buffer)"""
    import torch
    t = torch.full((M, N + pad), -7.0, dtype=getattr(torch, dt), device="cuda")
    return t[:, :N], t


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("form", FORMS)
def test_whole_numbers(gpu, shape, form):
    import torch
    (M, N, K), (op, kind, tB) = shape, form
    A = whole(M, K, 2, 0, kind, PAD)
    B = [whole(*((N, K) if tB else (K, N)), 2, i, kind, PAD) for i in range(1, 3 if op == "gated" else 2)]
    one = torch.ones(max(M, N), device="cuda")
    bufs = []
    new = lambda pad, dt: bufs.append(out(M, N, pad, dt)) or bufs[-1][0]  # noqa: E731
    x = product(A, B[0], tB)
    if op == "gated":
        C, g, u = new(8, "float32"), new(3, "bfloat16"), new(24, "bfloat16")
        bias = (torch.arange(N, device="cuda") % 5 - 2).float()
        if kind == "i8":
            gpu.run_gated_i8(A, one[:M], B[0], one[:N], B[1], one[:N], C, transB=tB, act="relu", bias_u=bias, g=g, u=u)
        else:
            gpu.run_gated(A, *B, C, transB=tB, act="relu", bias_u=bias, g=g, u=u)
        y = product(A, B[1], tB) + bias
        torch.cuda.synchronize()
        assert torch.equal(C, x.clamp(min=0) * y)
        assert torch.equal(g, x.bfloat16()) and torch.equal(u, y.bfloat16())
    elif op == "dgated":
        g, u = whole(M, N, 2, 3, pad=8), whole(M, N, 2, 4, pad=1)
        dg, du, h = new(16, "float32"), new(4, "float32"), new(5, "bfloat16")
        sg, su = (torch.full((N + 8,), -7.0, device="cuda") for _ in range(2))
        gpu.run_dgated(A, B[0], g, u, dg, du, transB=tB, act="relu", h=h, dbias_g=sg[:N], dbias_u=su[:N])
        on = (g > 0).float()
        wg, wu = x * u.float() * on, x * g.float() * on
        torch.cuda.synchronize()
        assert torch.equal(dg, wg) and torch.equal(du, wu) and torch.equal(h.float(), g.float() * on * u.float())
        for s, w in ((sg, wg), (su, wu)):
            assert w.abs().double().sum(0).max() < 2 ** 24
            assert torch.equal(s[:N].double(), w.double().sum(0)) and (s[N:] == -7).all()
    else:
        R, C = whole(M, N, 100, 2, pad=1), new(8, "bfloat16")
        gpu.run_i8(A, one[:M], B[0], one[:N], C, transB=tB, act="relu", residual=R, beta=2.0)
        torch.cuda.synchronize()
        assert torch.equal(C, (x.clamp(min=0) + 2.0 * R.float()).bfloat16())
    assert all((t[:, N:] == -7).all() for _, t in bufs)


@pytest.mark.parametrize("form", [f for f in FORMS if f[0] != "gated"])
def test_operands_of_many_megabytes(gpu, form):
    """G and U, or an fp32 residual, of more than 128 MB: 256 x 256 tiles read them past the caches."""
    import torch
    (op, kind, tB), (M, N, K) = form, (5003, 7696, 272)
    assert any(p.splits == 1 and "_pp_m256n256" in p.kernel for p in plan(*form, M, N, K, sums=op == "dgated", pad=PAD))
    A, B = whole(M, K, 2, 0, kind, PAD), whole(*((N, K) if tB else (K, N)), 2, 1, kind, PAD)
    x = product(A, B, tB)
    if op == "dgated":
        g, u = whole(M, N, 2, 3, pad=8), whole(M, N, 2, 4, pad=1)
        (dg, dgb), (du, dub), s = out(M, N, 1, "float32"), out(M, N, 3, "float32"), torch.empty(2, N, device="cuda")
        gpu.run_dgated(A, B, g, u, dg, du, transB=tB, act="relu", dbias_g=s[0], dbias_u=s[1])
        on = (g > 0).float()
        wg, wu = x * u.float() * on, x * g.float() * on
        torch.cuda.synchronize()
        assert torch.equal(dg, wg) and torch.equal(du, wu)
        assert torch.equal(s[0].double(), wg.double().sum(0)) and torch.equal(s[1].double(), wu.double().sum(0))
        assert (dgb[:, N:] == -7).all() and (dub[:, N:] == -7).all()
    else:
        one, R = torch.ones(max(M, N), device="cuda"), whole(M, N, 100, 2, pad=1).float()
        C, buf = out(M, N, 8, "float32")
        gpu.run_i8(A, one[:M], B, one[:N], C, transB=tB, act="relu", residual=R[:, :N], beta=2.0)
        torch.cuda.synchronize()
        assert torch.equal(C, x.clamp(min=0) + 2.0 * R[:, :N]) and (buf[:, N:] == -7).all()
