"""The gated and 8-bit integer operators on the GPU against the float64 oracle (oracle/gated.py).

Bounds, as for the MLP-block operators: U = 2^-24 is the fp32 unit; a bf16 output is allowed 2^-8 of
its value (half a step of it), an fp32 one 2^-22 (its half step is 2^-24).  A product's fp32 sum of K
terms is allowed 2 U sqrt(K) S (S the sum of the terms' magnitudes: the probabilistic scale, twice),
later operations 2 U of their operands.  A sum of 8-bit integers is exact: its conversion, its two
factors and the bias are four roundings of U each.  An activation has slope at most 1.2 and is evaluated
to EVAL (1 + |z|), its slope too.  Column sums are bounded by their terms' own errors plus U times the
terms' magnitudes times the longest chain of additions (rows).
"""
import numpy as np
import pytest

from oracle import gated, mlp
from test_gpu_mlp import DT, EVAL, U, dev, host, out_buffer, padding_untouched, within

pytestmark = pytest.mark.gpu

# few rows, widths of no whole eight, K of no whole 16 bytes, tiles' edges, splits, whole tiles
SHAPES = [(1, 8, 8), (1, 40, 64), (2, 33, 96), (3, 17, 5), (5, 64, 272), (13, 96, 208), (16, 512, 512), (17, 128, 1008),
          (33, 72, 32), (64, 64, 64), (65, 129, 71), (100, 304, 128), (127, 264, 512), (200, 1, 48), (257, 528, 304),
          (300, 512, 96), (512, 768, 320), (513, 272, 1024), (1, 1, 1), (40, 136, 8192), (1000, 2064, 528)]


def matrix(rng, rows, cols, kind, pad=0):
    """Random values of an operand type, rows of cols + pad: (device view, values)."""
    import torch
    if kind == "i8":
        v = rng.integers(-128, 128, (rows, cols + pad)).astype(np.int8)
        return torch.from_numpy(v).cuda()[:, :cols], v[:, :cols]
    t, v = dev(rng.standard_normal((rows, cols + pad)), kind)
    return t[:, :cols], v[:, :cols]


def vector(rng, n, kind="f32", positive=False):
    v = rng.standard_normal(n)
    t, v = dev(np.exp(v) * 1e-3 if positive else v, kind)
    return t, v.reshape(n)


def stored(rng, M, N, pad=0):
    t, v = dev(2.0 * rng.standard_normal((M, N + pad)), "bf16")
    return t[:, :N], v[:, :N]


def close(got, want, err, kind, what):
    within(host(got), want, DT[kind] * np.abs(want) + err + 2 * U * np.abs(want), what)


def gated_case(gpu, seed, M, N, K, tB, in_kind, out_kind, act, bias_kind=None, keep="gu", pads=(0, 0, 0), alpha=0.75,
               wide=False):
    """run_gated, or run_gated_i8 for "i8".  wide: both weights side by side in one buffer."""
    import torch
    rng = np.random.default_rng(seed)
    pa, pc, pz = pads
    A, Av = matrix(rng, M, K, in_kind, pa)
    shape = (N, K) if tB else (K, N)
    if wide:
        both, bv = matrix(rng, *((2 * N, K) if tB else (K, 2 * N)), in_kind, pa)
        cut = (slice(0, N), slice(N, 2 * N))
        (Bg, Bgv), (Bu, Buv) = (((both[c], bv[c]) if tB else (both[:, c], bv[:, c])) for c in cut)
    else:
        (Bg, Bgv), (Bu, Buv) = matrix(rng, *shape, in_kind, pa), matrix(rng, *shape, in_kind, pa)
    bg = bu = bgv = buv = None
    if bias_kind:
        bg, bgv = vector(rng, N, bias_kind)
        bu, buv = vector(rng, N, bias_kind)
    C, whole = out_buffer(M, N, out_kind, pc)
    g, gw = out_buffer(M, N, "bf16", pz) if "g" in keep else (None, None)
    u, uw = out_buffer(M, N, "bf16", pz) if "u" in keep else (None, None)
    if in_kind == "i8":
        (sa, sav), (sg, sgv), (su, suv) = vector(rng, M, positive=True), vector(rng, N, positive=True), vector(rng, N, positive=True)
        # factors that bring the products to about 1
        sav, sa = sav / 2, sa / 2
        gpu.run_gated_i8(A, sa, Bg, sg, Bu, su, C, transB=tB, act=act, bias_g=bg, bias_u=bu, g=g, u=u)
        G, Uv = gated.product_i8(Av, sav, Bgv, sgv, tB)[0], gated.product_i8(Av, sav, Buv, suv, tB)[0]
        G, Uv = G + (bgv if bias_kind else 0), Uv + (buv if bias_kind else 0)
        H = mlp.act(G, act) * Uv
        eg, eu = (4 * U * (np.abs(z) + 2 * (np.abs(b) if bias_kind else 0)) + 1e-30 for z, b in ((G, bgv), (Uv, buv)))
    else:
        gpu.run_gated(A, Bg, Bu, C, transB=tB, alpha=alpha, act=act, bias_g=bg, bias_u=bu, g=g, u=u)
        H, G, Uv, Sg, Su = gated.run_gated(Av, Bgv, Buv, alpha, act, bgv, buv, tB)
        eg, eu = (2 * U * (np.sqrt(K) * S + np.abs(z) + (np.abs(b) if bias_kind else 0)) + 1e-30
                  for S, z, b in ((Sg, G, bgv), (Su, Uv, buv)))
    torch.cuda.synchronize()
    what = f"{(M, N, K)} tB={tB} {in_kind}->{out_kind} {act} bias={bias_kind} keep={keep}"
    a, ea = np.abs(mlp.act(G, act)), 1.2 * eg + EVAL * (act != "none") * (1 + np.abs(G))
    close(C, H, np.abs(Uv) * ea + a * eu + ea * eu, out_kind, what)
    padding_untouched(whole, N, -77.0)
    for t, w, want, e in ((g, gw, G, eg), (u, uw, Uv, eu)):
        if t is not None:
            close(t, want, e, "bf16", what + ": kept")
            padding_untouched(w, N, -77.0)
    return C, g, u


def dgated_case(gpu, seed, M, N, K, tB, in_kind, out_kind, act, restore=True, sums="gu", pads=(0, 0, 0), alpha=0.5):
    import torch
    rng = np.random.default_rng(seed)
    pa, pc, pz = pads
    A, Av = matrix(rng, M, K, in_kind, pa)
    B, Bv = matrix(rng, *((N, K) if tB else (K, N)), in_kind, pa)
    (g, gv), (u, uv) = stored(rng, M, N, pz), stored(rng, M, N, pz)
    (dg, dgw), (du, duw) = out_buffer(M, N, out_kind, pc), out_buffer(M, N, out_kind, pc)
    h, hw = out_buffer(M, N, "bf16", pz) if restore else (None, None)
    sg = torch.full((N,), float("nan"), device="cuda:0") if "g" in sums else None
    su = torch.full((N,), float("nan"), device="cuda:0") if "u" in sums else None
    gpu.run_dgated(A, B, g, u, dg, du, transB=tB, alpha=alpha, act=act, h=h, dbias_g=sg, dbias_u=su)
    torch.cuda.synchronize()
    dG, dU, H, P, S = gated.run_dgated(Av, Bv, alpha, act, gv, uv, tB)
    ev = EVAL * (act != "none") * (1 + np.abs(gv))
    eP = 2 * U * (np.sqrt(K) * S + np.abs(P)) + 1e-30
    eG = np.abs(uv) * (1.2 * eP + ev * np.abs(P)) + 4 * U * np.abs(dG)
    eU = np.abs(mlp.act(gv, act)) * eP + ev * np.abs(P) + 4 * U * np.abs(dU)
    what = f"{(M, N, K)} tB={tB} {in_kind}->{out_kind} {act} restore={restore} sums={sums}"
    for t, w, want, e, s, n in ((dg, dgw, dG, eG, sg, "dG"), (du, duw, dU, eU, su, "dU")):
        close(t, want, e, out_kind, what + ": " + n)
        padding_untouched(w, N, -77.0)
        if s is not None:
            within(host(s), want.sum(0), e.sum(0) + U * M * np.abs(want).sum(0), what + ": sums of " + n)
    if restore:
        close(h, H, np.abs(uv) * ev + 2 * U * np.abs(H), "bf16", what + ": H")
        padding_untouched(hw, N, -77.0)
    return dg, du, h, sg, su


def i8_case(gpu, seed, M, N, K, tB, out_kind, act, bias_kind=None, res=False, pads=(0, 0, 0), beta=-0.5, in_place=False):
    import torch
    rng = np.random.default_rng(seed)
    pa, pc, _ = pads
    A, Av = matrix(rng, M, K, "i8", pa)
    B, Bv = matrix(rng, *((N, K) if tB else (K, N)), "i8", pa)
    (sa, sav), (sb, sbv) = vector(rng, M, positive=True), vector(rng, N, positive=True)
    bias, biasv = vector(rng, N, bias_kind) if bias_kind else (None, 0.0)
    C, whole = out_buffer(M, N, out_kind, pc)
    R = Rv = None
    if res:
        R, Rv = dev(rng.standard_normal((M, N + pc)), out_kind)
        R, Rv = R[:, :N], Rv[:, :N]
        if in_place:
            C.copy_(R)
            R = C
    gpu.run_i8(A, sa, B, sb, C, transB=tB, act=act, bias=bias, residual=R, beta=beta)
    torch.cuda.synchronize()
    P = gated.product_i8(Av, sav, Bv, sbv, tB)[0]
    Z = P + biasv
    want = mlp.act(Z, act) + (beta * Rv if res else 0)
    err = 1.2 * (4 * U * (np.abs(P) + np.abs(biasv)) + 1e-30) + EVAL * (act != "none") * (1 + np.abs(Z))
    err = err + 2 * U * (np.abs(want) + (abs(beta) * np.abs(Rv) if res else 0))
    close(C, want, err, out_kind, f"{(M, N, K)} tB={tB} i8->{out_kind} {act} bias={bias_kind} res={res}")
    padding_untouched(whole, N, -77.0)
    return C


ACT_OF = lambda i: mlp.ACTS[i % 5]  # noqa: E731
KINDS = ["bf16", "e4m3", "i8"]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("tB", [0, 1])
@pytest.mark.parametrize("kind", KINDS)
def test_run_gated(gpu, shape, tB, kind):
    i = SHAPES.index(shape) * 2 + tB + 3 * KINDS.index(kind)
    gated_case(gpu, i, *shape, tB, kind, ["bf16", "f32"][i % 2], ACT_OF(i), [None, "f32", "bf16"][i % 3],
               ["", "gu", "g", "u"][i % 4])
    gated_case(gpu, i, *shape, tB, kind, ["f32", "bf16"][i % 2], ACT_OF(i + 3), ["f32", None, None][i % 3],
               ["gu", ""][i % 2], wide=True)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("tB", [0, 1])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_run_dgated(gpu, shape, tB, kind):
    i = SHAPES.index(shape) * 2 + tB + 3 * KINDS.index(kind)
    dgated_case(gpu, i, *shape, tB, kind, ["bf16", "f32"][i % 2], ACT_OF(i), i % 3 != 0, ["gu", "", "g", "u"][i % 4])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("tB", [0, 1])
def test_run_i8(gpu, shape, tB):
    i = SHAPES.index(shape) * 2 + tB
    i8_case(gpu, i, *shape, tB, ["bf16", "f32"][i % 2], ACT_OF(i), [None, "f32", "bf16"][i % 3], i % 2 == 0)
    i8_case(gpu, i, *shape, tB, ["f32", "bf16"][i % 2], ACT_OF(i + 2), ["bf16", None, "f32"][i % 3], i % 2 == 1,
            in_place=True)


@pytest.mark.parametrize("act", mlp.ACTS)
@pytest.mark.parametrize("shape", [(7, 208, 128), (256, 256, 256), (384, 640, 512), (24, 128, 4096)])
def test_every_activation(gpu, shape, act):
    for kind in KINDS:
        gated_case(gpu, 7, *shape, 1, kind, "bf16", act, "f32")
    dgated_case(gpu, 8, *shape, 0, "bf16", "bf16", act)
    dgated_case(gpu, 8, *shape, 1, "e4m3", "f32", act)
    i8_case(gpu, 9, *shape, 1, "bf16", act, "f32", True)


# strides past the rows, 16-byte aligned or not
@pytest.mark.parametrize("pads", [(16, 8, 32), (1, 3, 5), (0, 1, 0)])
@pytest.mark.parametrize("shape", [(5, 96, 80), (130, 272, 144), (300, 528, 256)])
@pytest.mark.parametrize("tB", [0, 1])
def test_strides(gpu, shape, pads, tB):
    for kind in KINDS:
        gated_case(gpu, 31, *shape, tB, kind, "bf16", "silu", "bf16", pads=pads)
    dgated_case(gpu, 32, *shape, tB, "bf16", "bf16", "gelu", pads=pads)
    i8_case(gpu, 33, *shape, tB, "bf16", "silu", "bf16", True, pads=pads)


# widths and K that are whole 16-byte pieces but no whole tiles; widths past the last whole eight
# with operands that the MFMA kernels take
@pytest.mark.parametrize("shape", [(70, 83, 96), (9, 131, 512), (150, 1037, 1040), (321, 515, 2576), (2, 2050, 256)])
def test_widths_of_no_whole_eight(gpu, shape):
    for kind in KINDS:
        gated_case(gpu, 41, *shape, 1, kind, "bf16", "gelu_tanh", "f32")
    dgated_case(gpu, 42, *shape, 1, "bf16", "f32", "silu")
    dgated_case(gpu, 42, *shape, 1, "e4m3", "bf16", "silu", sums="u")
    i8_case(gpu, 43, *shape, 1, "bf16", "none", "f32", True)


# more 256 x 256 tiles than CUs and not whole rounds of them
@pytest.mark.parametrize("shape", [(1300, 6544, 320), (13104, 656, 320)])
@pytest.mark.parametrize("tB", [0, 1])
def test_many_tiles(gpu, shape, tB):
    M, N, K = shape
    for kind in KINDS:
        gated_case(gpu, 70, M, N, K, tB, kind, "bf16", "silu", "f32", pads=(16, 8, 32), alpha=0.1)
    for kind in ("bf16", "e4m3"):
        dgated_case(gpu, 72, M, 2 * N, K, tB, kind, "bf16", "relu", alpha=0.1)
    i8_case(gpu, 73, M, 2 * N, K, tB, "f32", "none", None, True)


def test_gradients_in_place(gpu):
    """dG over G and dU over U: the bits of separate buffers."""
    import torch
    for M, N, K in ((3, 40, 24), (64, 128, 512), (300, 520, 256), (65, 129, 71), (40, 136, 8192)):
        rng = np.random.default_rng(5)
        A, B = matrix(rng, M, K, "bf16")[0], matrix(rng, N, K, "bf16")[0]
        g, u = stored(rng, M, N)[0], stored(rng, M, N)[0]
        dg, du = torch.empty_like(g), torch.empty_like(u)
        h = [torch.empty_like(g), torch.empty_like(g)]
        gpu.run_dgated(A, B, g, u, dg, du, transB=1, act="gelu", h=h[0])
        gpu.run_dgated(A, B, g, u, g, u, transB=1, act="gelu", h=h[1])
        torch.cuda.synchronize()
        assert torch.equal(g, dg) and torch.equal(u, du) and torch.equal(*h)


@pytest.mark.parametrize("shape", [(300, 520, 256), (65, 129, 71), (40, 136, 8192), (1000, 2064, 528), (20, 264, 512)])
def test_the_same_bits_every_run(gpu, shape):
    import torch
    first = None
    for _ in range(3):
        dg, du, h, sg, su = dgated_case(gpu, 23, *shape, 1, "bf16", "bf16", "silu")
        c, g, u = gated_case(gpu, 24, *shape, 1, "bf16", "bf16", "silu", "f32")
        out = [t.float().cpu().numpy() for t in (dg, du, h, sg, su, c, g, u)]
        first = first or out
        assert all(np.array_equal(x, y) for x, y in zip(out, first))


def test_products_without_terms(gpu):
    """K = 0 and alpha = 0: the epilogue of a zero product; empty outputs; sums over no rows."""
    import torch
    M, N = 37, 72
    (bg, bgv), (bu, buv) = vector(np.random.default_rng(0), N), vector(np.random.default_rng(1), N)
    want = np.broadcast_to(mlp.act(bgv, "silu") * buv, (M, N))
    bound = EVAL * (1 + np.abs(bgv)) * np.abs(buv) + 4 * U * np.abs(want)
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    for dt in (torch.bfloat16, torch.float8_e4m3fn):
        C, _ = out_buffer(M, N, "f32")
        gpu.run_gated(e(M, 0, dt=dt), e(0, N, dt=dt), e(0, N, dt=dt), C, bias_g=bg, bias_u=bu)
        torch.cuda.synchronize()
        within(host(C), want, bound, "K = 0")
    A, _ = dev(np.ones((M, 16)), "bf16")
    B, _ = dev(np.full((16, N), np.inf), "bf16")
    C.fill_(-1)
    gpu.run_gated(A, B, B, C, alpha=0.0, bias_g=bg, bias_u=bu)
    torch.cuda.synchronize()
    within(host(C), want, bound, "alpha = 0")
    i8 = torch.int8
    sa, sb = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    gpu.run_gated_i8(e(M, 0, dt=i8), sa, e(0, N, dt=i8), sb, e(0, N, dt=i8), sb, C.fill_(-1), bias_g=bg, bias_u=bu)
    torch.cuda.synchronize()
    within(host(C), want, bound, "K = 0")
    gpu.run_i8(e(M, 0, dt=i8), sa, e(0, N, dt=i8), sb, C.fill_(-1), bias=bg)
    torch.cuda.synchronize()
    assert np.array_equal(host(C), np.broadcast_to(bgv, (M, N)))
    z = e(0, N)
    sg, su = torch.full((N,), 5.0, device="cuda"), torch.full((N,), 5.0, device="cuda")
    gpu.run_dgated(A[:0], B, z, z, z, z, dbias_g=sg, dbias_u=su)
    torch.cuda.synchronize()
    assert (sg == 0).all() and (su == 0).all()
    su.fill_(5.0)
    gpu.run_dgated(A[:0], B, z, z, z, z, dbias_u=su)
    gpu.run_gated(A[:0], B, B, z)
    gpu.run_gated(A, B[:, :0], B[:, :0], e(M, 0))
    torch.cuda.synchronize()
    assert (su == 0).all()


def test_nan_and_inf_stay_in_their_places(gpu):
    """A row of A with NaN or Inf reaches its own row only, a column of B its own column."""
    import torch
    for M, N, K in ((40, 96, 64), (300, 512, 128), (5, 64, 512)):
        rng = np.random.default_rng(5)
        x = rng.standard_normal((M, K))
        x[2, 7] = np.nan
        A = dev(x, "bf16")[0]
        w = np.abs(rng.standard_normal((N, K))) + 0.1
        Bg = dev(w, "bf16")[0]
        w2 = w.copy()
        w2[3, 5] = np.inf
        Bu = dev(w2, "bf16")[0]
        C, _ = out_buffer(M, N, "bf16")
        for act in mlp.ACTS:
            gpu.run_gated(A, Bg, Bu, C, transB=1, act=act)
            torch.cuda.synchronize()
            c = host(C)
            assert np.isnan(c[2]).all(), act
            assert not np.isfinite(c[:, 3]).any() or act == "relu", act
            assert np.isfinite(np.delete(np.delete(c, 2, 0), 3, 1)).all(), act
        g = dev(rng.standard_normal((M, N)), "bf16")[0]
        u = g.clone()
        u[4, 6] = float("nan")
        (dg, _), (du, _) = out_buffer(M, N, "bf16"), out_buffer(M, N, "bf16")
        gpu.run_dgated(dev(w[:1].repeat(M, 0), "bf16")[0], Bg, g, u, dg, du, transB=1)
        torch.cuda.synchronize()
        assert np.isnan(host(dg)[4, 6]) and np.isfinite(host(du)).all()
        assert np.isfinite(host(dg)).sum() == M * N - 1


# ------------------------------------------------------------------------------ 8-bit integers

def test_sums_are_exact(gpu):
    """Codes at their ends over the longest K: the sum itself, in 32 bits."""
    import torch
    K = 131071
    ones = lambda n: torch.ones(n, device="cuda:0")  # noqa: E731
    for K in (131071, 131056, 4096):
        for M, N in ((1, 8), (3, 33), (70, 64)):
            A = torch.full((M, K), -128, dtype=torch.int8, device="cuda:0")
            B = torch.full((N, K), -128, dtype=torch.int8, device="cuda:0")
            B[1] = 127
            C, _ = out_buffer(M, N, "f32")
            gpu.run_i8(A, ones(M), B, ones(N), C, transB=1)
            torch.cuda.synchronize()
            want = np.full((M, N), np.float32(16384 * K))
            want[:, 1] = np.float32(-128 * 127 * K)
            assert np.array_equal(host(C), want), (M, N, K)


@pytest.mark.parametrize("shape", [(1, 40, 64), (20, 520, 512), (70, 264, 2064), (513, 1040, 272), (33, 24, 16384)])
@pytest.mark.parametrize("tB", [0, 1])
def test_i8_products_are_exact(gpu, shape, tB):
    """Factors of 1 and sums under 2^24: every element is the whole number itself."""
    import torch
    M, N, K = shape
    rng = np.random.default_rng(3)
    a, b, b2 = (rng.integers(-20, 21, s).astype(np.int8) for s in ((M, K), (N, K), (N, K)))
    t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    one = lambda n: torch.ones(n, device="cuda:0")  # noqa: E731
    B, B2 = (t(x if tB else x.T) for x in (b, b2))
    C, _ = out_buffer(M, N, "f32")
    gpu.run_i8(t(a), one(M), B, one(N), C, transB=tB)
    torch.cuda.synchronize()
    p, p2 = a.astype(np.int64) @ b.T, a.astype(np.int64) @ b2.T
    assert np.array_equal(host(C), p)
    gpu.run_gated_i8(t(a), one(M), B, one(N), B2, one(N), C, transB=tB, act="relu")
    torch.cuda.synchronize()
    assert np.array_equal(host(C), (np.maximum(p, 0).astype(np.float32) * p2.astype(np.float32)).astype(np.float64))


def test_i8_factors_of_nan(gpu):
    """A row that could not be quantised (factor NaN) gives NaN, and its neighbours do not."""
    import torch
    for M in (5, 100):
        rng = np.random.default_rng(1)
        A, B = matrix(rng, M, 256, "i8")[0], matrix(rng, 64, 256, "i8")[0]
        sa, sb = torch.ones(M, device="cuda"), torch.ones(64, device="cuda")
        sa[3] = float("nan")
        C, _ = out_buffer(M, 64, "bf16")
        for call in (lambda: gpu.run_i8(A, sa, B, sb, C, transB=1),
                     lambda: gpu.run_gated_i8(A, sa, B, sb, B, sb, C, transB=1, act="relu")):
            call()
            torch.cuda.synchronize()
            c = host(C)
            assert np.isnan(c[3]).all() and np.isfinite(np.delete(c, 3, 0)).all()


def test_refusals(gpu):
    import dense_blas3_gemm_amd as d
    import torch
    e = lambda *s: torch.empty(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    K = 131072
    C = torch.full((2, 8), -1.0, device="cuda")
    sa, sb = torch.ones(2, device="cuda"), torch.ones(8, device="cuda")
    with pytest.raises(d.GemmError, match="NOT_SUPPORTED"):
        gpu.run_i8(e(2, K), sa, e(8, K), sb, C, transB=1)
    with pytest.raises(d.GemmError, match="NOT_SUPPORTED"):
        gpu.run_gated_i8(e(2, K), sa, e(8, K), sb, e(8, K), sb, C, transB=1)
    A, B = torch.ones(2, 16, dtype=torch.bfloat16, device="cuda"), torch.ones(16, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(d.GemmError, match="NOT_SUPPORTED"):
        gpu.run_gated(A, B, B, C, alpha=float("inf"))
    with pytest.raises(ValueError, match="cuda:0"):
        gpu.run_gated(A, B.cpu(), B, C)
    with pytest.raises(ValueError, match="cuda:0"):
        gpu.run_gated(A, B, B.cpu(), C)
    torch.cuda.synchronize()
    assert (C == -1).all()
    # through the C-ABI: what the binding cannot send
    lib, h = d.load_library(), gpu.handle
    ptr = lambda t: t.data_ptr()  # noqa: E731
    import ctypes
    gate, ep = d.Gate(act=4), d.Epilogue()
    ok = lambda **kw: {**dict(tb=0, M=2, N=8, K=16, lda=16, ldb=8, ldb2=8, ldc=8, act=4, dtype=d.BF16_F32, A=ptr(A), B=ptr(B),  # noqa: E731
                              B2=ptr(B), C=ptr(C), ep=ctypes.byref(gate)), **kw}
    run = lambda a: lib.gemm_run_gated(h, a["tb"], a["M"], a["N"], a["K"], 1.0, a["A"], a["lda"], a["B"], a["ldb"], a["B2"],  # noqa: E731
                                       a["ldb2"], a["ep"], a["C"], a["ldc"], a["dtype"])
    assert run(ok()) == 0
    for bad in (dict(tb=2), dict(M=-1), dict(K=2 ** 31), dict(lda=15), dict(ldb=7), dict(ldb2=7), dict(ldc=7), dict(B2=0),
                dict(A=0), dict(C=0), dict(ep=None), dict(dtype=d.E4M3_E4M3), dict(ep=ctypes.byref(d.Gate(act=5))),
                dict(ep=ctypes.byref(d.Gate(act=1, bias_u=ptr(sb), bias_type=2))),
                dict(ep=ctypes.byref(d.Gate(act=1, g=ptr(C), ld_g=7)))):
        assert run(ok(**bad)) == 1, bad
    A8, B8 = e(2, 16), e(16, 8)
    run8 = lambda sa=ptr(sa), sb=ptr(sb), ct=1, ep=ep: lib.gemm_run_i8(  # noqa: E731
        h, 0, 2, 8, 16, ptr(A8), 16, sa, ptr(B8), 8, sb, ctypes.byref(ep), ptr(C), 8, ct)
    assert run8() == 0
    assert run8(sa=0) == run8(sb=0) == run8(ct=2) == run8(ep=d.Epilogue(z_kind=1)) == 1
    assert run8(ep=d.Epilogue(residual=ptr(C), ld_residual=8, beta=float("nan"))) == 2
    q = lambda rows=2, cols=8, t=1, ld=8, s=ptr(sa): lib.gemm_quantize_i8(h, rows, cols, ptr(C), ld, t, ptr(A8), 16, s)  # noqa: E731
    assert q() == 0 and q(rows=0) == 0
    assert q(rows=-1) == q(cols=2 ** 31) == q(t=2) == q(ld=7) == q(s=0) == 1
    torch.cuda.synchronize()


QUANT = [(1, 1), (1, 7), (1, 8), (1, 5120), (3, 33), (5, 511), (4, 512), (6, 513), (64, 100), (5, 1024), (3, 1025), (5, 2049),
         (130, 4100), (700, 96), (1031, 40), (2, 8200), (3, 13696), (2, 20480), (1, 40001), (600, 2048), (2, 70000)]


def quantized(gpu, x, pad=0):
    import torch
    M, N = x.shape
    q = torch.full((M, N + pad), 0x5A, dtype=torch.int8, device="cuda:0")
    s = torch.full((M,), -1.0, device="cuda:0")
    gpu.quantize_i8(x, q[:, :N], s)
    torch.cuda.synchronize()
    assert (q[:, N:] == 0x5A).all(), "written past the rows"
    return q[:, :N].cpu().numpy(), s.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("shape", QUANT)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 3])
def test_quantize_i8(gpu, shape, kind, pad):
    M, N = shape
    rng = np.random.default_rng(N)
    x, xv = dev(np.ldexp(rng.standard_normal((M, N + pad)), rng.integers(-30, 30, (M, 1))), kind)
    q, s = quantized(gpu, x[:, :N], pad)
    rows = np.unique(np.r_[0:min(M, 4), M - 1])
    want, scale = gated.quantize_i8(xv[rows, :N])
    assert np.array_equal(q[rows], want)
    # one rounding
    assert (np.abs(s[rows] - scale) <= U * scale).all()
    top = np.abs(xv[:, :N]).max(1)
    assert (np.abs(s - top / 127) <= U * top / 127).all()
    assert (np.abs(q * (top / 127)[:, None] - xv[:, :N]) <= (0.5 + 1e-9) * (top / 127)[:, None]).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_quantize_i8_middles(gpu, kind):
    """Values at the middles between codes and one step of their type beside them, at every largest
    magnitude of a binade; tiny and huge rows."""
    import torch
    tops = np.arange(128, 256) / 128.0
    k = np.arange(-127, 127) + 0.5
    x = k[None, :] * tops[:, None] / 127.0
    x = torch.from_numpy(np.concatenate([x, tops[:, None]], 1))
    x = x.to(torch.bfloat16 if kind == "bf16" else torch.float32)
    step = 2.0 ** -7 if kind == "bf16" else 2.0 ** -23
    near = [x, (x.double() * (1 + step)).to(x.dtype), (x.double() * (1 - step)).to(x.dtype)]
    for n in near:
        n[:, -1] = x[:, -1]
    x = torch.cat(near, 1)
    for e in (0, -110, -126, 100, 120):
        y = (x.double() * 2.0 ** e).to(x.dtype)
        q, s = quantized(gpu, y.cuda())
        want, scale = gated.quantize_i8(y.double().numpy())
        assert np.array_equal(q, want), e
        assert (np.abs(s - scale) <= U * scale + 2.0 ** -150).all()


def test_quantize_i8_special_rows(gpu):
    import torch
    for kind in (torch.bfloat16, torch.float32):
        for N in (5, 300, 3000, 20000):
            x = torch.randn(6, N).to(kind)
            x[0] = 0
            x[1, N // 2], x[2, N - 1], x[3, 0] = float("nan"), float("inf"), float("-inf")
            x[4] = -0.0
            q, s = quantized(gpu, x.cuda())
            assert (q[:5] == 0).all() and s[0] == 0 and s[4] == 0 and np.isnan(s[1:4]).all()
            assert np.abs(q[5]).max() == 127
    # the smallest numbers of all, and no columns
    x = torch.full((1, 9), 2.0 ** -149)
    q, s = quantized(gpu, x.cuda())
    assert (q == 127).all()
    q, s = quantized(gpu, torch.empty(3, 0, device="cuda"))
    assert (s == 0).all()
    gpu.quantize_i8(torch.empty(0, 8, device="cuda"), torch.empty(0, 8, dtype=torch.int8, device="cuda"),
                    torch.empty(0, device="cuda"))


# ------------------------------------------------------------------- streams, graphs, devices

def test_captured_and_replayed(gpu):
    """A chain of the operators captured into a graph, replayed between eager calls on the same
    handle: every replay gives the eager bits for the inputs of the day."""
    import torch
    M, N, K = 300, 528, 4096
    rng = np.random.default_rng(9)
    A, Bg, Bu, Wd = (matrix(rng, *s, "bf16")[0] for s in ((M, K), (N, K), (N, K), (N, K)))
    wg, wu = torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, K, dtype=torch.int8, device="cuda")
    sg, su = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    gpu.quantize_i8(Bg, wg, sg)
    gpu.quantize_i8(Bu, wu, su)
    e = lambda *s, dt=torch.bfloat16: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731

    def chain(o):
        gpu.run_gated(A, Bg, Bu, o[0], transB=1, alpha=0.02, g=o[1], u=o[2])
        gpu.run_dgated(A, Wd, o[1], o[2], o[3], o[4], transB=1, alpha=0.02, h=o[5], dbias_g=o[6], dbias_u=o[7])
        gpu.quantize_i8(A, o[8], o[9])
        gpu.run_gated_i8(o[8], o[9], wg, sg, wu, su, o[10], transB=1)

    def buffers():
        return [e(M, N) for _ in range(6)] + [e(N, dt=torch.float32) for _ in range(2)] + [
            e(M, K, dt=torch.int8), e(M, dt=torch.float32), e(M, N)]
    out, want = buffers(), buffers()
    chain(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        chain(out)
    for i in range(4):
        A.copy_(torch.from_numpy(rng.standard_normal((M, K))).to(torch.bfloat16))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        chain(want)
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x.float(), y.float()), i


def test_on_another_stream(gpu):
    """Enqueued on torch's current stream: inputs that it makes are seen without a wait."""
    import torch
    M, N, K = 64, 256, 1024
    rng = np.random.default_rng(2)
    A, Bg, Bu = (matrix(rng, *s, "bf16")[0] for s in ((M, K), (N, K), (N, K)))
    C, ref = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    gpu.run_gated(A, Bg, Bu, ref, transB=1)
    x = torch.zeros_like(A)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(5):
            big = big @ big * 1e-3
        x.copy_(A)
        gpu.run_gated(x, Bg, Bu, C, transB=1)
        x.zero_()
    torch.cuda.synchronize()
    assert torch.equal(C, ref)
