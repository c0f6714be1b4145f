"""The gated operators where 256 x 256 tiles split K between workgroups: few rows, wide outputs, and a
K of no whole tiles, so that the last part is shorter.  And weights, outputs and stored operands whose
strides differ from each other.  Whole numbers with every sum under 2^24, so that any order of
additions gives the exact sum, and what follows it is compared bit by bit."""
import pytest

pytestmark = pytest.mark.gpu

CASES = [(255, 8624, 7600), (165, 10224, 14800), (361, 7360, 5232), (1, 8624, 7600)]


def whole(rows, cols, span, seed, dt="bf16", pad=0):
    import torch
    r = torch.Generator("cuda").manual_seed(seed)
    t = torch.randint(-span, span + 1, (rows, cols + pad), generator=r, device="cuda").float()
    return t.to({"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}[dt])[:, :cols]


def product(A, B, tB):
    """fp32: exact here."""
    b = B.float()
    return A.float() @ (b.t() if tB else b)


@pytest.mark.parametrize("shape", CASES)
@pytest.mark.parametrize("tB", [0, 1])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_gated(gpu, shape, tB, kind):
    import torch
    M, N, K = shape
    A = whole(M, K, 2, 0, kind, 16)
    Bg, Bu = (whole(*((N, K) if tB else (K, N)), 2, i, kind, 16 * i) for i in (1, 2))
    C = torch.full((M, N + 8), -7.0, device="cuda")
    g = torch.full((M, N + 3), -7.0, dtype=torch.bfloat16, device="cuda")
    u = torch.full((M, N + 24), -7.0, dtype=torch.bfloat16, device="cuda")
    if kind == "i8":
        one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
        gpu.run_gated_i8(A, one(M), Bg, one(N), Bu, one(N), C[:, :N], transB=tB, act="relu", g=g[:, :N], u=u[:, :N])
    else:
        gpu.run_gated(A, Bg, Bu, C[:, :N], transB=tB, act="relu", g=g[:, :N], u=u[:, :N])
    torch.cuda.synchronize()
    x, y = product(A, Bg, tB), product(A, Bu, tB)
    assert torch.equal(C[:, :N], x.clamp(min=0) * y)
    assert torch.equal(g[:, :N], x.bfloat16()) and torch.equal(u[:, :N], y.bfloat16())
    assert all((t[:, N:] == -7).all() for t in (C, g, u))


@pytest.mark.parametrize("shape", [(1129, 4144, 5488), (255, 12304, 7600), (700, 5200, 9040)])
@pytest.mark.parametrize("tB", [0, 1])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_dgated(gpu, shape, tB, kind):
    import torch
    M, N, K = shape
    A, B = whole(M, K, 2, 0, kind, 16), whole(*((N, K) if tB else (K, N)), 2, 1, kind)
    g, u = whole(M, N, 2, 2, pad=8), whole(M, N, 2, 3, pad=1)
    e = lambda pad, dt=torch.bfloat16: torch.full((M, N + pad), -7.0, dtype=dt, device="cuda")  # noqa: E731
    dg, du, h = e(16, torch.float32), e(4, torch.float32), e(5)
    sg, su = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    gpu.run_dgated(A, B, g, u, dg[:, :N], du[:, :N], transB=tB, act="relu", h=h[:, :N], dbias_g=sg, dbias_u=su)
    torch.cuda.synchronize()
    p = product(A, B, tB)
    on = (g > 0).float()
    x, y = p * u.float() * on, p * g.float() * on
    assert torch.equal(dg[:, :N], x) and torch.equal(du[:, :N], y)
    assert torch.equal(h[:, :N].float(), g.float() * on * u.float())
    assert x.abs().sum(0).max() < 2 ** 24 and y.abs().sum(0).max() < 2 ** 24
    assert torch.equal(sg, x.sum(0)) and torch.equal(su, y.sum(0))
    assert all((t[:, N:] == -7).all() for t in (dg, du, h))


@pytest.mark.parametrize("shape", [(149, 19472, 14512), (255, 12304, 15216), (700, 5200, 18064)])
@pytest.mark.parametrize("tB", [0, 1])
def test_i8(gpu, shape, tB):
    import torch
    M, N, K = shape
    A, B = whole(M, K, 2, 0, "i8", 16), whole(*((N, K) if tB else (K, N)), 2, 1, "i8")
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    R = whole(M, N, 100, 2, pad=1)
    C = torch.full((M, N + 8), -7.0, dtype=torch.bfloat16, device="cuda")
    gpu.run_i8(A, one(M), B, one(N), C[:, :N], transB=tB, act="relu", residual=R, beta=2.0)
    torch.cuda.synchronize()
    want = (product(A, B, tB).clamp(min=0) + 2.0 * R.float()).bfloat16()
    assert torch.equal(C[:, :N], want)
    assert (C[:, N:] == -7).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_i8_residual_of_many_megabytes(gpu, kind):
    """A residual past half the caches, beside the output and over it."""
    import torch
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[kind]
    M, N, K = 8200, 8208, 528
    A, B = whole(M, K, 2, 0, "i8"), whole(N, K, 2, 1, "i8")
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    C = whole(M, N, 100, 2, pad=8).to(dt)
    R, out = C.clone(), torch.empty_like(C)
    gpu.run_i8(A, one(M), B, one(N), out, transB=1, residual=R, beta=-1.0)
    gpu.run_i8(A, one(M), B, one(N), C, transB=1, residual=C, beta=-1.0)
    torch.cuda.synchronize()
    want = (product(A, B, 1) - R.float()).to(dt)
    assert torch.equal(out, want) and torch.equal(C, want)


def test_gradients_of_many_megabytes(gpu):
    """G and U past half the caches, in place and not."""
    import torch
    M, N, K = 5000, 7688, 256
    A, B = whole(M, K, 2, 0), whole(N, K, 2, 1)
    g, u = whole(M, N, 2, 2), whole(M, N, 2, 3)
    dg, du, h = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g)
    p, on = product(A, B, 1), (g > 0).float()
    x, y = (p * u.float() * on).bfloat16(), (p * g.float() * on).bfloat16()
    gpu.run_dgated(A, B, g, u, dg, du, transB=1, act="relu", h=h)
    torch.cuda.synchronize()
    assert torch.equal(dg, x) and torch.equal(du, y) and torch.equal(h.float(), g.float() * on * u.float())
    gpu.run_dgated(A, B, g, u, g, u, transB=1, act="relu")
    torch.cuda.synchronize()
    assert torch.equal(g, x) and torch.equal(u, y)


def test_two_handles_on_two_streams():
    """Split products and column sums side by side: each handle has its own workspace."""
    import torch
    import dense_blas3_gemm_amd as d
    hs = [d.Gemm(0), d.Gemm(0)]
    try:
        M, N, K = 255, 1040, 8208
        A, B = [whole(M, K, 2, i) for i in (0, 1)], [whole(N, K, 2, i) for i in (2, 3)]
        g, u = [whole(M, N, 2, i) for i in (4, 5)], [whole(M, N, 2, i) for i in (6, 7)]
        out = [[torch.empty(M, N, device="cuda") for _ in range(3)] + [torch.empty(N, device="cuda") for _ in range(2)]
               for _ in range(2)]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for _ in range(20):
            for h, s, a, b, gg, uu, o in zip(hs, streams, A, B, g, u, out):
                with torch.cuda.stream(s):
                    h.run_gated(a, b, b, o[0], transB=1, act="relu")
                    h.run_dgated(a, b, gg, uu, o[1], o[2], transB=1, act="relu", dbias_g=o[3], dbias_u=o[4])
        torch.cuda.synchronize()
        for a, b, gg, uu, o in zip(A, B, g, u, out):
            p, on = product(a, b, 1), (gg > 0).float()
            x, y = p * uu.float() * on, p * gg.float() * on
            assert torch.equal(o[0], p.clamp(min=0) * p) and torch.equal(o[1], x) and torch.equal(o[2], y)
            assert torch.equal(o[3], x.sum(0)) and torch.equal(o[4], y.sum(0))
    finally:
        for h in hs:
            h.close()


def test_captured_odd_and_split(gpu):
    """Split tiles, left columns and column sums replayed between eager calls of the same handle."""
    import torch
    M, N, K = 255, 1045, 8208
    A, B = whole(M, K, 2, 0), whole(N, K, 2, 1)
    g, u = whole(M, N, 2, 2), whole(M, N, 2, 3)
    mk = lambda: [torch.empty(M, N, device="cuda") for _ in range(3)] + [torch.empty(N, device="cuda") for _ in range(2)]  # noqa: E731
    out, want = mk(), mk()

    def run(o):
        gpu.run_gated(A, B, B, o[0], transB=1, act="relu")
        gpu.run_dgated(A, B, g, u, o[1], o[2], transB=1, act="relu", dbias_g=o[3], dbias_u=o[4])
    run(want)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run(out)
    for i in range(4):
        A.copy_(whole(M, K, 2, 10 + i))
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        run(want)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want)), i
    p = product(A, B, 1)
    assert torch.equal(out[0], p.clamp(min=0) * p)
