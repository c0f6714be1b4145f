"""The MLP-block operators on the GPU against the float64 oracle (oracle/mlp.py), through the
binding and the C-ABI.

Bounds.  u = 2^-24 is the fp32 unit; a bf16 output is allowed 2^-8 of its value (twice the rounding),
an fp32 one 2^-22.  A product's fp32 sum of K terms is allowed 2 u sqrt(K) S (S the sum of the terms'
magnitudes: the probabilistic scale, twice), later additions 2 u of their operands.  An activation has
slope at most 1.2 and is evaluated to EVAL (1 + |z|): the erf form is good to 1.5e-7, the exponential
and the reciprocal to 2^-23 each, and a handful of fp32 roundings follow.  Column sums are bounded by
their terms' own errors plus u times the terms' magnitudes times the longest chain of additions (rows).
"""
import numpy as np
import pytest

import gemm_inputs as gi
import oracle
from gpu_util import to_device, to_host
from oracle import mlp

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EVAL = 1e-6
DT = {"bf16": 2.0 ** -8, "f32": 2.0 ** -22}


def dev(x, kind):
    """float64 values -> (device tensor, its values as float64)."""
    import torch
    x32 = np.ascontiguousarray(x, dtype=np.float32)
    if kind == "f32":
        return torch.from_numpy(x32).cuda(), x32.astype(np.float64)
    bits = gi.f32_to_bf16_bits(x32) if kind == "bf16" else gi.f32_to_e4m3_bits(x32)
    return to_device(bits, kind), oracle.decode(bits, kind).reshape(x.shape)


def host(t):
    import torch
    return t.to(torch.float32).cpu().numpy().astype(np.float64)


def torch_type(kind):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[kind]


def out_buffer(M, N, kind, pad=0, fill=-77.0):
    """An M x N view of rows of N + pad elements, all `fill`, and the whole buffer."""
    import torch
    whole = torch.full((M, N + pad), fill, dtype=torch_type(kind), device="cuda:0")
    return whole[:, :N], whole


def mx_buffers(M, N, pad=0):
    import torch
    q = torch.full((M, N + pad), 0x5A, dtype=torch.uint8, device="cuda:0")
    s = torch.full((M, (N + 31) // 32 + pad), 0x5A, dtype=torch.uint8, device="cuda:0")
    return q[:, :N], s[:, :(N + 31) // 32], q, s


def padding_untouched(whole, N, fill):
    w = whole[:, N:].float().cpu().numpy()
    assert np.all(w == fill), "written past the rows"


def mx_values(q, s):
    return mlp.from_mx(oracle.decode(q.cpu().numpy().reshape(-1), "e4m3").reshape(tuple(q.shape)), s.cpu().numpy())


def within(got, want, bound, what):
    assert np.isfinite(got).all(), what
    bad = np.abs(got - want) > bound
    if bad.any():
        i = np.unravel_index(np.argmax(np.abs(got - want) / bound), got.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside; worst at {i}: {got[i]} for {want[i]}, "
                             f"bound {bound[i]}")


def check_mx(q, s, Z, errZ, what):
    """Codes of values within errZ of Z: the scale is that of some such values, each element is
    within half a step of E4M3 at that scale (saturated above 448)."""
    M, N = Z.shape
    sc = s.cpu().numpy().astype(np.int64)
    pad = -N % 32
    lo = np.pad(np.maximum(np.abs(Z) - errZ, 0.0), ((0, 0), (0, pad))).reshape(M, -1, 32).max(2)
    hi = np.pad(np.abs(Z) + errZ, ((0, 0), (0, pad))).reshape(M, -1, 32).max(2)
    def code(a):
        e = np.frexp(a)[1] - 1 - 8 + 127
        return np.where(a > 0, np.clip(e, 0, 254), 0)
    assert ((code(lo) <= sc) & (sc <= code(hi))).all(), f"{what}: scales"
    step = np.repeat(np.ldexp(1.0, sc - 127), 32, axis=1)[:, :N]  # the scale itself
    v = mx_values(q, s)
    a = np.abs(Z) / step
    half = np.maximum(np.ldexp(1.0, np.frexp(a)[1] - 1 - 4), 2.0 ** -10)  # half of 2^(floor(log2 a) - 3)
    bound = np.where(a + errZ / step > 448.0, np.maximum(a - 448.0, 0) + 16.0, half) * step + errZ * 2
    within(v, Z, bound, what)


# ------------------------------------------------------------------------- products

SHAPES = [(1, 8, 8), (1, 40, 64), (2, 33, 96), (3, 17, 5), (5, 64, 264), (13, 96, 200), (16, 512, 512), (17, 128, 1000),
          (33, 72, 24), (64, 64, 64), (65, 129, 71), (100, 300, 128), (127, 264, 512), (200, 1, 40), (257, 520, 304),
          (300, 512, 96), (512, 768, 320), (513, 264, 1024), (1, 1, 1)]
ACT_OF = lambda i: mlp.ACTS[i % 5]  # noqa: E731


def act_case(gpu, i, M, N, K, trans, in_kind, out_kind, act, bias_kind, res, z_kind, pads=(0, 0, 0), alpha=0.75,
             beta=-0.5, ints=False, in_place=False):
    import torch
    rng = np.random.default_rng(1000 + i)
    tA, tB = trans
    pa, pc, pz = pads
    draw = (lambda *s: rng.integers(-4, 5, s).astype(np.float64)) if ints else (lambda *s: rng.standard_normal(s))
    a_shape, b_shape = ((K, M) if tA else (M, K)), ((N, K) if tB else (K, N))
    A, Av = dev(draw(a_shape[0], a_shape[1] + pa), in_kind)
    B, Bv = dev(draw(b_shape[0], b_shape[1] + pa), in_kind)
    A, Av, B, Bv = A[:, :a_shape[1]], Av[:, :a_shape[1]], B[:, :b_shape[1]], Bv[:, :b_shape[1]]
    bias = biasv = R = Rv = z = zs = None
    if bias_kind:
        bias, biasv = dev(draw(N), bias_kind)
        biasv = biasv.reshape(N)
    C, whole = out_buffer(M, N, out_kind, pc)
    if res:
        R, Rv = dev(draw(M, N + pc), out_kind)
        R, Rv = R[:, :N], Rv[:, :N]
        if in_place:
            C.copy_(R)
            R = C
    if z_kind == "bf16":
        z, zwhole = out_buffer(M, N, "bf16", pz)
    elif z_kind == "mx":
        z, zs, zwhole, swhole = mx_buffers(M, N, pz)
    gpu.run_act(A, B, C, transA=tA, transB=tB, alpha=alpha, act=act, bias=bias, residual=R, beta=beta, z=z,
                z_scales=zs)
    torch.cuda.synchronize()
    want, Z, S = mlp.run_act(Av, Bv, alpha, act, biasv, Rv, beta, tA, tB)
    errZ = 2 * U * (np.sqrt(K) * S + np.abs(Z) + (np.abs(biasv) if bias_kind else 0)) + 1e-30
    bound = (DT[out_kind] * np.abs(want) + 1.2 * errZ + EVAL * (act != "none") * (1 + np.abs(Z)) +
             2 * U * (np.abs(want) + (abs(beta) * np.abs(Rv) if res else 0)))
    what = f"{(M, N, K)} {trans} {in_kind}->{out_kind} {act} bias={bias_kind} res={res} z={z_kind}"
    within(host(C), want, bound, what)
    padding_untouched(whole, N, -77.0)
    if z_kind == "bf16":
        within(host(z), Z, DT["bf16"] * np.abs(Z) + errZ, what + ": Z")
        padding_untouched(zwhole, N, -77.0)
    elif z_kind == "mx":
        check_mx(z, zs, Z, errZ, what + ": Z")
        padding_untouched(zwhole, N, 0x5A)
        padding_untouched(swhole, (N + 31) // 32, 0x5A)
    return z, zs, Z


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("trans", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_run_act(gpu, shape, trans):
    i = SHAPES.index(shape) * 4 + trans[0] * 2 + trans[1]
    for j, (kind, out) in enumerate([("bf16", "bf16"), ("bf16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32")]):
        k = i + 3 * j
        act_case(gpu, k, *shape, trans, kind, out, ACT_OF(k), [None, "f32", "bf16"][k % 3], (k // 2) % 2 == 0,
                 ["none", "mx", "bf16"][(k // 3) % 3])


@pytest.mark.parametrize("act", mlp.ACTS)
@pytest.mark.parametrize("z_kind", ["none", "bf16", "mx"])
@pytest.mark.parametrize("shape", [(7, 200, 128), (256, 256, 256), (384, 640, 512)])
def test_run_act_every_activation(gpu, shape, act, z_kind):
    act_case(gpu, 7, *shape, (0, 1), "bf16", "bf16", act, "f32", True, z_kind)


# strides past the rows, 16-byte aligned or not
@pytest.mark.parametrize("pads", [(8, 8, 32), (1, 3, 5), (0, 1, 0)])
@pytest.mark.parametrize("shape", [(5, 96, 72), (130, 264, 136), (300, 520, 256)])
def test_run_act_strides(gpu, shape, pads):
    for j, z in enumerate(("mx", "bf16")):
        act_case(gpu, 31 + j, *shape, (0, j), "bf16", "bf16", "silu", "bf16", True, z, pads=pads)


# one shape of every kernel that the shape-driven choice has for a product with an epilogue
@pytest.mark.parametrize("shape", [(1000, 2056, 520), (2048, 1536, 256), (700, 5120, 320)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_run_act_large_tiles(gpu, shape, kind):
    M, N, K = shape
    K = K // 16 * 16
    for j, (z, out) in enumerate((("mx", "bf16"), ("bf16", "f32"))):
        act_case(gpu, 50 + j, M, N // 16 * 16, K, (0, 1 - j), kind, out, "gelu_tanh", "f32", True, z)


def test_run_act_long_k_small_output(gpu):
    """Few output tiles and a long K: split products."""
    for M in (3, 40, 96):
        act_case(gpu, M, M, 128, 8192, (0, 1), "bf16", "bf16", "gelu", "f32", True, "mx", alpha=0.01)
        act_case(gpu, M, M, 136, 6144 + 8, (0, 0), "bf16", "f32", "silu", "f32", True, "bf16", alpha=0.01)


# E4M3 operands under 256 x 256 tiles: whole and ragged tiles, a K of one tile and less, a K
# that ends inside a tile, split and not
@pytest.mark.parametrize("shape", [(70, 80, 96), (65, 144, 2064), (130, 272, 4112), (150, 528, 1040), (320, 512, 112),
                                   (384, 1152, 2576), (72, 2048, 256), (272, 4096, 528)])
@pytest.mark.parametrize("trans", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_e4m3_small_tiles(gpu, shape, trans):
    M, N, K = shape
    if trans[0]:
        M = M // 16 * 16  # rows of whole 16-byte pieces
    i = 60 + trans[0] * 2 + trans[1]
    act_case(gpu, i, M, N, K, trans, "e4m3", "bf16", "gelu", "f32", True, "mx", alpha=0.02)
    act_case(gpu, i, M, N, K, trans, "e4m3", "f32", "silu", "bf16", False, "bf16", alpha=0.02)
    dact_case(gpu, i, M, N, K, trans, "bf16", "silu", "mx", in_kind="e4m3", alpha=0.02)


# more 256 x 256 tiles than CUs and not whole rounds of them: two launches, cut by columns or by
# rows, the second on other tiles
@pytest.mark.parametrize("shape", [(1300, 13088, 320), (13104, 1296, 320)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_products_in_two_launches(gpu, shape, kind):
    M, N, K = shape
    tB = int(kind == "e4m3")
    act_case(gpu, 70, M, N, K, (0, tB), kind, "bf16", "silu", "f32", True, "mx", pads=(16, 8, 32), alpha=0.1)
    act_case(gpu, 71, M, N, K, (int(M % 16 == 0), 1 - tB), kind, "f32", "none", "bf16", False, "bf16", alpha=0.1)
    dact_case(gpu, 72, M, N, K, (0, 1 - tB), "bf16", "relu", "mx", in_kind=kind, alpha=0.1)


def test_run_act_in_place_residual(gpu):
    for shape in ((3, 40, 24), (70, 132, 64), (256, 512, 128), (65, 129, 71)):
        act_case(gpu, 5, *shape, (0, 1), "bf16", "bf16", "gelu", "f32", True, "none", in_place=True, pads=(0, 8, 0))


@pytest.mark.parametrize("shape", [(2, 40, 64), (65, 129, 71), (130, 264, 512), (256, 512, 128), (40, 96, 4096),
                                   (9, 256, 512)])
def test_run_act_exact_codes(gpu, shape):
    """Integer operands: the fp32 sum is exact, so the codes and scales are the oracle's."""
    for tB in (0, 1):
        z, zs, Z = act_case(gpu, 3, *shape, (0, tB), "bf16", "f32", "none", "f32", False, "mx", alpha=1.0, ints=True)
        codes, scales = oracle.quantize_mx(Z)
        assert np.array_equal(zs.cpu().numpy(), scales)
        assert np.array_equal(z.cpu().numpy() & 0x7F, codes & 0x7F)  # the sign of zero aside
        nz = (codes & 0x7F) != 0
        assert np.array_equal(z.cpu().numpy()[nz], codes[nz])


def dact_case(gpu, i, M, N, K, trans, out_kind, act, z_kind, in_kind="bf16", pads=(0, 0, 0), dbias=True, alpha=0.5):
    import torch
    rng = np.random.default_rng(2000 + i)
    tA, tB = trans
    pa, pc, pz = pads
    a_shape, b_shape = ((K, M) if tA else (M, K)), ((N, K) if tB else (K, N))
    A, Av = dev(rng.standard_normal((a_shape[0], a_shape[1] + pa)), in_kind)
    B, Bv = dev(rng.standard_normal((b_shape[0], b_shape[1] + pa)), in_kind)
    A, Av, B, Bv = A[:, :a_shape[1]], Av[:, :a_shape[1]], B[:, :b_shape[1]], Bv[:, :b_shape[1]]
    z, zv = dev(2.0 * rng.standard_normal((M, N + pz)), "bf16")
    z, zv, zs = z[:, :N], zv[:, :N], None
    if z_kind == "mx":
        q, zs, _, _ = mx_buffers(M, N, pz)
        gpu.quantize_mx(z, q, zs)
        z, zv = q, mx_values(q, zs)
    C, whole = out_buffer(M, N, out_kind, pc)
    db = torch.full((N,), float("nan"), device="cuda:0") if dbias else None
    gpu.run_dact(A, B, C, z, z_scales=zs, transA=tA, transB=tB, alpha=alpha, act=act, dbias=db)
    torch.cuda.synchronize()
    D, sums, P, S = mlp.run_dact(Av, Bv, alpha, act, zv, tA, tB)
    errD = 1.2 * 2 * U * np.sqrt(K) * S + EVAL * (act != "none") * np.abs(P) * (1 + np.abs(zv)) + 4 * U * np.abs(D) + 1e-30
    what = f"{(M, N, K)} {trans} ->{out_kind} {act} z={z_kind}"
    within(host(C), D, errD + DT[out_kind] * np.abs(D), what)
    padding_untouched(whole, N, -77.0)
    if dbias:
        within(host(db), sums, errD.sum(0) + U * M * np.abs(D).sum(0), what + ": dbias")
    return C, db


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("trans", [(0, 0), (0, 1), (1, 0), (1, 1)])
def test_run_dact(gpu, shape, trans):
    i = SHAPES.index(shape) * 4 + trans[0] * 2 + trans[1]
    dact_case(gpu, i, *shape, trans, ["bf16", "f32"][i % 2], ACT_OF(i), ["mx", "bf16"][(i // 2) % 2])
    dact_case(gpu, i, *shape, trans, ["f32", "bf16"][i % 2], ACT_OF(i + 2), ["bf16", "mx"][(i // 2) % 2],
              in_kind="e4m3", dbias=i % 3 != 0)


@pytest.mark.parametrize("act", mlp.ACTS)
@pytest.mark.parametrize("z_kind", ["bf16", "mx"])
@pytest.mark.parametrize("shape", [(7, 200, 128), (300, 520, 256), (1000, 2056, 520), (40, 136, 8192)])
def test_run_dact_every_activation(gpu, shape, act, z_kind):
    dact_case(gpu, 11, *shape, (0, 1), "bf16", act, z_kind)


@pytest.mark.parametrize("pads", [(8, 8, 32), (1, 3, 5)])
def test_run_dact_strides(gpu, pads):
    for shape in ((5, 96, 72), (130, 264, 136), (300, 520, 256)):
        for z in ("mx", "bf16"):
            dact_case(gpu, 17, *shape, (0, 0), "bf16", "gelu", z, pads=pads)


@pytest.mark.parametrize("shape", [(300, 520, 256), (65, 129, 71), (40, 136, 8192), (1000, 2056, 520)])
def test_dbias_is_the_same_every_run(gpu, shape):
    import torch
    first = None
    for _ in range(3):
        C, db = dact_case(gpu, 23, *shape, (0, 1), "bf16", "silu", "mx")
        bits = (db.view(torch.int32).cpu().numpy(), C.view(torch.int16).cpu().numpy())
        first = first or bits
        assert np.array_equal(bits[0], first[0]) and np.array_equal(bits[1], first[1])


def test_products_without_terms(gpu):
    """K = 0 and alpha = 0: the epilogue of a zero product; empty outputs."""
    import torch
    M, N = 37, 72
    bias, biasv = dev(np.linspace(-3, 3, N), "f32")
    A, B = torch.empty(M, 0, dtype=torch.bfloat16, device="cuda"), torch.empty(0, N, dtype=torch.bfloat16, device="cuda")
    want = mlp.act(np.broadcast_to(biasv, (M, N)), "silu")
    C, _ = out_buffer(M, N, "f32")
    ep = _epilogue(act="silu", bias=bias)
    assert _raw_act(gpu, M, N, 0, 1.0, 0, 1, 0, N, ep, C) == 0
    torch.cuda.synchronize()
    within(host(C), want, EVAL * (1 + np.abs(want)), "K = 0")
    A, _ = dev(np.ones((M, 16)), "bf16")
    B, _ = dev(np.full((16, N), np.inf), "bf16")
    C.fill_(-1)
    gpu.run_act(A, B, C, alpha=0.0, act="silu", bias=bias)
    torch.cuda.synchronize()
    within(host(C), want, EVAL * (1 + np.abs(want)), "alpha = 0")
    db = torch.full((N,), 5.0, device="cuda")
    z, _ = dev(np.zeros((0, N)), "bf16")
    gpu.run_dact(A[:0], B, C[:0], z.reshape(0, N), act="relu", dbias=db)
    torch.cuda.synchronize()
    assert (db == 0).all()
    gpu.run_act(A[:0], B, C[:0], act="relu", bias=bias)


def test_nan_and_inf_stay_in_their_places(gpu):
    """A row of A with NaN or Inf reaches its own row of C and Z only."""
    import torch
    for M, N, K in ((40, 96, 64), (300, 512, 128), (5, 64, 512)):
        rng = np.random.default_rng(5)
        x = rng.standard_normal((M, K))
        x[2, 7], x[4, 3] = np.nan, np.inf
        A, Av = dev(x, "bf16")
        B, Bv = dev(np.abs(rng.standard_normal((N, K))) + 0.1, "bf16")
        C, _ = out_buffer(M, N, "bf16")
        z, zs, _, _ = mx_buffers(M, N)
        for act in mlp.ACTS:
            gpu.run_act(A, B, C, transB=1, act=act, z=z, z_scales=zs)
            torch.cuda.synchronize()
            c = host(C)
            assert np.isnan(c[2]).all() and np.isposinf(c[4]).all(), act
            assert np.isfinite(np.delete(c, [2, 4], 0)).all(), act
            q = z.cpu().numpy()
            assert ((q[2] & 0x7F) == 0x7F).all()  # NaN codes
            assert ((q[4] & 0x7F) == 0x7E).all()  # Inf saturates
            assert ((np.delete(q, [2, 4], 0) & 0x7F) != 0x7F).all()


# ------------------------------------------------------------- 8-bit checkpoints of activations

ROWS_COLS = [(1, 1), (1, 31), (1, 32), (1, 5120), (3, 33), (7, 257), (64, 100), (5, 2049), (130, 4100), (700, 96),
             (1031, 40)]


@pytest.mark.parametrize("shape", ROWS_COLS)
@pytest.mark.parametrize("pad", [0, 3])
def test_act_mx(gpu, shape, pad):
    import torch
    M, N = shape
    i = ROWS_COLS.index(shape)
    rng = np.random.default_rng(i)
    z, zv = dev(np.ldexp(rng.standard_normal((M, N + pad)), rng.integers(-12, 6, (M, 1))), "bf16")
    z, zv = z[:, :N], zv[:, :N]
    for act in mlp.ACTS:
        H, whole = out_buffer(M, N, "bf16", pad)
        q, s, qw, sw = mx_buffers(M, N, pad)
        gpu.act_mx(z, H, q, s, act=act)
        torch.cuda.synchronize()
        want = mlp.act(zv, act)
        within(host(H), want, DT["bf16"] * np.abs(want) + EVAL * (act != "none") * np.minimum(np.abs(zv), 1 + np.abs(zv)) + 1e-38, act)
        q2, s2, _, _ = mx_buffers(M, N, pad)
        gpu.quantize_mx(z, q2, s2)  # pinned against the oracle by its own tests
        assert torch.equal(q, q2) and torch.equal(s, s2)
        padding_untouched(whole, N, -77.0)
        padding_untouched(qw, N, 0x5A)
        padding_untouched(sw, (N + 31) // 32, 0x5A)


@pytest.mark.parametrize("shape", ROWS_COLS)
@pytest.mark.parametrize("pad", [0, 3])
def test_act_grad_mx(gpu, shape, pad):
    import torch
    M, N = shape
    rng = np.random.default_rng(ROWS_COLS.index(shape))
    z, _ = dev(2 * rng.standard_normal((M, N)), "bf16")
    q, s, _, _ = mx_buffers(M, N, pad)
    gpu.quantize_mx(z, q, s)
    zv = mx_values(q, s)
    dh, dv = dev(rng.standard_normal((M, N + pad)), "bf16")
    dh, dv = dh[:, :N], dv[:, :N]
    for act in mlp.ACTS:
        D, H = dv * mlp.slope(zv, act), mlp.act(zv, act)
        errD = EVAL * (act != "none") * np.abs(dv) * (1 + np.abs(zv)) + 2 * U * np.abs(D) + 1e-38
        errH = EVAL * (act != "none") * (1 + np.abs(zv)) + 1e-38
        for want_dz, want_db, want_h in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0)):
            dz, dzw = out_buffer(M, N, "bf16", pad) if want_dz else (None, None)
            h, hw = out_buffer(M, N, "bf16", pad) if want_h else (None, None)
            db = torch.full((N,), float("nan"), device="cuda:0") if want_db else None
            gpu.act_grad_mx(q, s, act=act, dh=dh if want_dz or want_db else None, dz=dz, dbias=db, h=h)
            torch.cuda.synchronize()
            if want_dz:
                within(host(dz), D, DT["bf16"] * np.abs(D) + errD, act)
                padding_untouched(dzw, N, -77.0)
            if want_db:
                within(host(db), D.sum(0), errD.sum(0) + U * M * np.abs(D).sum(0), act + ": dbias")
            if want_h:
                within(host(h), H, DT["bf16"] * np.abs(H) + errH, act + ": h")
                padding_untouched(hw, N, -77.0)
    inplace = dh.clone()
    dz, _ = out_buffer(M, N, "bf16")
    gpu.act_grad_mx(q, s, act="gelu", dh=inplace, dz=dz)
    gpu.act_grad_mx(q, s, act="gelu", dh=inplace, dz=inplace)
    torch.cuda.synchronize()
    assert torch.equal(inplace, dz)


def test_act_grad_mx_extremes(gpu):
    """The format's ends: scale 0 (2^-127), the largest finite codes, a NaN scale, huge arguments."""
    import torch
    q = torch.tensor([[0x7E] * 32 + [0xFE] * 32 + [0x01] * 32 + [0x30] * 32], dtype=torch.uint8, device="cuda")
    s = torch.tensor([[190, 190, 0, 255]], dtype=torch.uint8, device="cuda")
    dh = torch.ones((1, 128), dtype=torch.bfloat16, device="cuda")
    for act in mlp.ACTS[1:]:
        dz, h = torch.empty_like(dh), torch.empty_like(dh)
        gpu.act_grad_mx(q, s, act=act, dh=dh, dz=dz, h=h)
        torch.cuda.synchronize()
        dz, h = host(dz)[0], host(h)[0]
        big = 448.0 * 2.0 ** 63
        assert (dz[:32] == 1).all() and (np.abs(h[:32] / big - 1) < 2.0 ** -8).all(), act
        assert (dz[32:64] == 0).all() and (h[32:64] == 0).all(), act
        assert (np.abs(dz[64:96] - (1.0 if act == "relu" else 0.5)) < 2.0 ** -8).all(), act
        assert (np.abs(h[64:96]) < 1e-38).all(), act
        assert np.isnan(dz[96:]).all() and np.isnan(h[96:]).all(), act
    db = torch.full((128,), 3.0, device="cuda")
    gpu.act_grad_mx(q[:0], s[:0], act="relu", dh=dh[:0], dbias=db)
    torch.cuda.synchronize()
    assert (db == 0).all()


# ------------------------------------------------------------------------------ layer norm

NORM_SHAPES = [(1, 1), (1, 2), (3, 7), (1, 64), (2, 65), (5, 256), (4, 511), (3, 1024), (2, 2047), (130, 96), (1, 5120),
               (9, 4099), (700, 130), (3, 8192), (2, 8200), (2, 16384), (2, 20480), (2, 32768), (1, 40001), (2100, 264),
               (4100, 72)]


def norm_inputs(rng, M, N, kind, pad):
    x = rng.standard_normal((M, N + pad)) * rng.uniform(0.5, 2.0, (M, 1)) + 2 * rng.standard_normal((M, 1))
    t, v = dev(x, kind)
    return t[:, :N], v[:, :N]


def chain(N):
    """Longest run of fp32 additions in a row's sum: a lane takes 1/64 of the row, then a tree."""
    return -(-N // 64) + 16


@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("pad", [0, 1])
def test_layernorm(gpu, shape, pad):
    import torch
    M, N = shape
    for i, (xk, yk, wk) in enumerate([("bf16", "bf16", "f32"), ("f32", "bf16", "bf16"), ("f32", "f32", "f32"),
                                      ("bf16", "f32", None)]):
        rng = np.random.default_rng(17 * NORM_SHAPES.index(shape) + i)
        x, xv = norm_inputs(rng, M, N, xk, pad)
        g = gv = b = bv = None
        if wk:
            g, gv = dev(1 + 0.2 * rng.standard_normal(N), wk)
            b, bv = dev(rng.standard_normal(N), wk)
            gv, bv = gv.reshape(N), bv.reshape(N)
        if i == 2:
            b = bv = None
        y, whole = out_buffer(M, N, yk, pad)
        mean, rstd = torch.full((M,), float("nan"), device="cuda"), torch.full((M,), float("nan"), device="cuda")
        if i != 1:
            gpu.layernorm(x, y, gamma=g, beta=b, eps=1e-3, mean=mean, rstd=rstd)
        else:
            gpu.layernorm(x, y, gamma=g, beta=b, eps=1e-3)
        torch.cuda.synchronize()
        want, mu, r = mlp.layernorm(xv, gv, bv, eps=1e-3)
        d = chain(N)
        e_mu = d * U * np.abs(xv).mean(1)
        # the squares carry twice the error of x - mu, whose mean square is at most 1 / r^2
        e_r = r * (0.5 * (d + 6) * U + r * r * e_mu * (np.abs(xv - mu[:, None]).mean(1) + e_mu) + 4 * U)
        if i != 1:
            within(host(mean), mu, e_mu + 1e-30, "mean")
            within(host(rstd), r, e_r, "rstd")
        gabs = np.abs(gv) if wk else 1.0
        err = gabs * ((e_mu[:, None] + 2 * U * np.abs(xv)) * r[:, None] + np.abs(xv - mu[:, None]) * (e_r[:, None] + 2 * U * r[:, None]))
        err = err + 2 * U * (np.abs(want) + (np.abs(bv) if bv is not None else 0))
        within(host(y), want, err + DT[yk] * np.abs(want) + 1e-30, f"{shape} {xk}->{yk} {wk}")
        padding_untouched(whole, N, -77.0)


@pytest.mark.parametrize("shape", NORM_SHAPES)
@pytest.mark.parametrize("pad", [0, 1])
def test_layernorm_grad(gpu, shape, pad):
    import torch
    M, N = shape
    for i, (xk, yk, wk) in enumerate([("bf16", "bf16", "f32"), ("f32", "bf16", "bf16"), ("f32", "f32", None),
                                      ("bf16", "f32", "f32")]):
        rng = np.random.default_rng(19 * NORM_SHAPES.index(shape) + i)
        x, xv = norm_inputs(rng, M, N, xk, pad)
        dy, dyv = dev(rng.standard_normal((M, N + pad)), yk)
        dy, dyv = dy[:, :N], dyv[:, :N]
        g = gv = res = resv = None
        if wk:
            g, gv = dev(1 + 0.2 * rng.standard_normal(N), wk)
            gv = gv.reshape(N)
        if i % 2:
            res, resv = dev(rng.standard_normal((M, N + pad)), xk)
            res, resv = res[:, :N], resv[:, :N]
        _, mu, r = mlp.layernorm(xv, eps=1e-3)
        mean, mu = dev(mu, "f32")
        rstd, r = dev(r, "f32")
        dx, whole = out_buffer(M, N, xk, pad)
        dg, db = torch.full((N,), float("nan"), device="cuda"), torch.full((N,), float("nan"), device="cuda")
        if i == 3:  # the residual's gradient in place
            dx.copy_(res)
            res = dx
        gpu.layernorm_grad(dy, x, mean, rstd, dx, gamma=g, dgamma=dg if i != 2 else None, dbeta=db if i else None,
                           residual=res)
        torch.cuda.synchronize()
        want, dgv, dbv = mlp.layernorm_grad(dyv, xv, mu, r, gv, resv)
        n = np.abs(xv - mu[:, None]) * r[:, None]
        e_n = (2 * U * (np.abs(xv) + np.abs(mu[:, None])) * r[:, None]) + 2 * U * n
        ga = np.abs(dyv) * (np.abs(gv) if wk else 1.0)
        d = chain(N) + 4
        c2 = (ga * n).mean(1)[:, None]
        e_c1, e_c2 = d * U * ga.mean(1)[:, None], d * U * c2 + (ga * e_n).mean(1)[:, None]
        err = r[:, None] * (2 * U * ga + e_c1 + n * e_c2 + e_n * c2 + 4 * U * (ga + ga.mean(1)[:, None] + n * c2))
        err = err + 2 * U * (np.abs(want) + (np.abs(resv) if resv is not None else 0))
        what = f"{shape} x {xk} dy {yk} gamma {wk}"
        within(host(dx), want, err + DT[xk] * np.abs(want) + 1e-30, what)
        padding_untouched(whole, N, -77.0)
        if i != 2:
            within(host(dg), dgv, (np.abs(dyv) * e_n).sum(0) + (M + 4) * U * (np.abs(dyv) * n).sum(0) + 1e-30, what + ": dgamma")
        if i:
            within(host(db), dbv, (M + 2) * U * np.abs(dyv).sum(0) + 1e-30, what + ": dbeta")


def test_layernorm_in_place_and_edges(gpu):
    import torch
    for M, N in ((3, 96), (2, 5120), (1, 40001)):
        x = torch.randn(M, N, device="cuda").bfloat16()
        y = torch.empty_like(x)
        gpu.layernorm(x, y)
        gpu.layernorm(x, x)
        torch.cuda.synchronize()
        assert torch.equal(x, y)
    # a constant row: y = beta, rstd = 1 / sqrt(eps); with eps = 0 the definition's 0 * inf
    x = torch.full((2, 200), 3.0, device="cuda")
    y, r = torch.empty_like(x), torch.empty(2, device="cuda")
    gpu.layernorm(x, y, eps=0.25, rstd=r)
    torch.cuda.synchronize()
    assert (y == 0).all() and (r == 2).all()
    gpu.layernorm(x, y, eps=0.0, rstd=r)
    torch.cuda.synchronize()
    assert torch.isnan(y).all() and torch.isinf(r).all()
    # a large mean: the deviations are taken before they are squared
    x = 1e4 + torch.randn(3, 777, device="cuda")
    y = torch.empty_like(x)
    gpu.layernorm(x, y, eps=1e-6)
    torch.cuda.synchronize()
    want = mlp.layernorm(host(x), eps=1e-6)[0]
    assert np.abs(host(y) - want).max() < 777 * U * 1e4 / 10
    # NaN stays in its row
    x = torch.randn(5, 333, device="cuda")
    x[2, 17] = float("nan")
    y = torch.empty_like(x)
    gpu.layernorm(x, y)
    torch.cuda.synchronize()
    assert torch.isnan(y[2]).all() and torch.isfinite(y[[0, 1, 3, 4]]).all()
    # no rows: the weights' gradients are zeros
    dg, db = torch.full((64,), 2.0, device="cuda"), torch.full((64,), 2.0, device="cuda")
    e = torch.empty((0, 64), device="cuda")
    gpu.layernorm_grad(e, e, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"), e, dgamma=dg, dbeta=db)
    torch.cuda.synchronize()
    assert (dg == 0).all() and (db == 0).all()


@pytest.mark.parametrize("shape", [(700, 130), (2100, 264), (300, 5120)])
def test_layernorm_grad_is_the_same_every_run(gpu, shape):
    import torch
    M, N = shape
    torch.manual_seed(0)
    x, dy = torch.randn(M, N, device="cuda").bfloat16(), torch.randn(M, N, device="cuda").bfloat16()
    mean, rstd = x.float().mean(1), 1 / x.float().std(1)
    got = []
    for _ in range(3):
        dx, dg, db = torch.empty_like(x), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
        gpu.layernorm_grad(dy, x, mean, rstd, dx, dgamma=dg, dbeta=db)
        got.append((dx, dg, db))
    torch.cuda.synchronize()
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_offsets_past_32_bits(gpu):
    """Rows a GiB of elements apart: element offsets pass 2^31."""
    import torch
    ld = 1 << 30
    for N in (100, 5120):
        buf = torch.empty(3 * ld, dtype=torch.bfloat16, device="cuda")
        x = buf.view(3, ld)[:, :N]
        x.copy_(torch.randn(3, N, device="cuda"))
        y, small = torch.empty(3, N, device="cuda", dtype=torch.bfloat16), x.clone()
        gpu.layernorm(small, y)
        gpu.layernorm(x, x)
        torch.cuda.synchronize()
        assert torch.equal(x, y)
        z, zs = torch.empty(3, N, dtype=torch.uint8, device="cuda"), torch.empty(3, (N + 31) // 32, dtype=torch.uint8, device="cuda")
        h, z2, zs2 = torch.empty_like(y), torch.empty_like(z), torch.empty_like(zs)
        gpu.act_mx(x, h, z, zs, act="gelu")
        want = torch.empty_like(h)
        gpu.act_mx(y, want, z2, zs2, act="gelu")
        torch.cuda.synchronize()
        assert torch.equal(h, want) and torch.equal(z, z2) and torch.equal(zs, zs2)
        # C and the residual of a product
        A, B = torch.randn(3, 64, device="cuda").bfloat16(), torch.randn(N, 64, device="cuda").bfloat16()
        r = x.clone()
        gpu.run_act(A, B, y, transB=1, act="gelu", residual=r)
        gpu.run_act(A, B, x, transB=1, act="gelu", residual=x)
        torch.cuda.synchronize()
        assert torch.equal(x, y)
        del buf, x
        torch.cuda.empty_cache()


# ------------------------------------------------------------------- streams, graphs, refusals

def test_calls_follow_the_current_stream(gpu):
    """Inputs made on a side stream, the call on that stream, the result read there."""
    import torch
    s = torch.cuda.Stream()
    M, N, K = 300, 520, 256
    A0, B0 = torch.randn(M, K, device="cuda").bfloat16(), torch.randn(N, K, device="cuda").bfloat16()
    torch.cuda.synchronize()
    want = torch.empty(M, N, device="cuda", dtype=torch.bfloat16)
    gpu.run_act(A0, B0, want, transB=1, act="gelu")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(5):
            A = torch.zeros_like(A0)
            for _ in range(20):
                A = A + A0 * 0.05  # keeps the stream busy before the call
            A.copy_(A0)
            C, y = torch.empty_like(want), torch.empty_like(want)
            gpu.run_act(A, B0, C, transB=1, act="gelu")
            gpu.layernorm(C, y)
    s.synchronize()
    assert torch.equal(C, want)


def test_graph_replays(gpu):
    """The block's calls in a graph, replayed between eager work."""
    import torch
    torch.manual_seed(1)
    M, H = 96, 512
    x = torch.randn(M, H, device="cuda").bfloat16()
    w = torch.randn(H, H, device="cuda").bfloat16() * H ** -0.5
    b = torch.randn(H, device="cuda")
    u, h, out = (torch.empty_like(x) for _ in range(3))
    z, zs = torch.empty(M, H, dtype=torch.uint8, device="cuda"), torch.empty(M, H // 32, dtype=torch.uint8, device="cuda")
    db, mean, rstd = torch.empty(H, device="cuda"), torch.empty(M, device="cuda"), torch.empty(M, device="cuda")

    def step():
        gpu.layernorm(x, u, gamma=b, eps=1e-5, mean=mean, rstd=rstd)
        gpu.run_act(u, w, h, transB=1, act="gelu_tanh", bias=b, z=z, z_scales=zs)
        gpu.run_act(h, w, out, transB=1, residual=x)
        gpu.run_dact(out, w, h, z, z_scales=zs, act="gelu_tanh", dbias=db)

    step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for i in range(4):
        x.copy_(torch.randn(M, H, device="cuda"))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (u, h, out, z, zs, db, mean, rstd)]
        for t in (u, h, out, db, mean, rstd):
            t.fill_(float("nan"))
        z.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip((u, h, out, z, zs, db, mean, rstd), want)), i


def _epilogue(**kw):
    import dense_blas3_gemm_amd as d
    ep = d.Epilogue(d.ACTS[kw.get("act", "none")])
    if kw.get("bias") is not None:
        ep.bias, ep.bias_type = kw["bias"].data_ptr(), d.TYPE_F32
    return ep


def _raw_act(gpu, M, N, K, alpha, A, lda, B, ldb, ep, C):
    import ctypes
    import dense_blas3_gemm_amd as d
    gpu._bind(C)
    return gpu.lib.gemm_run_act(gpu.handle, 0, 0, M, N, K, alpha, A, lda, B, ldb, ctypes.byref(ep), C.data_ptr(),
                                C.stride(0), d.BF16_F32)


def test_refusals_of_the_c_abi(gpu):
    """Bad arguments are rejected and nothing is written."""
    import ctypes
    import torch
    import dense_blas3_gemm_amd as d
    lib, h = gpu.lib, gpu.handle
    M, N, K = 32, 64, 32
    buf = torch.full((64, 64), 7.0, device="cuda")
    p = buf.data_ptr()
    gpu._bind(buf)

    def act(h=h, ep=True, **kw):
        a = dict(tA=0, tB=0, M=M, N=N, K=K, alpha=1.0, A=p, lda=K, B=p, ldb=N, C=p, ldc=N, dtype=d.BF16_F32)
        e = d.Epilogue()
        for k, v in kw.items():
            if k in a:
                a[k] = v
            else:
                setattr(e, k, v)
        return lib.gemm_run_act(h, a["tA"], a["tB"], a["M"], a["N"], a["K"], a["alpha"], a["A"], a["lda"], a["B"],
                                a["ldb"], ctypes.byref(e) if ep else None, a["C"], a["ldc"], a["dtype"])

    assert act(h=None) == 3 and act(ep=False) == 1
    for kw in (dict(act=5), dict(act=-1), dict(tA=2), dict(M=-1), dict(lda=K - 1), dict(ldb=N - 1), dict(ldc=N - 1),
               dict(A=None), dict(C=None), dict(dtype=d.E4M3_E4M3), dict(dtype=d.MXE4M3_BF16), dict(dtype=99),
               dict(bias=p, bias_type=2), dict(residual=p, ld_residual=N - 1), dict(z_kind=3), dict(z_kind=-1),
               dict(z_kind=1, ld_z=N), dict(z_kind=1, z=p, ld_z=N - 1), dict(z_kind=2, z=p, ld_z=N, ld_z_scales=2),
               dict(z_kind=2, z=p, ld_z=N, z_scales=p, ld_z_scales=1)):
        assert act(**kw) == 1, kw
    assert act(alpha=float("nan")) == 2
    assert act(residual=p, ld_residual=N, beta=float("inf")) == 2
    dact = lambda h=h, act=1, kind=1, z=p, ldz=N, s=None, lds=0, C=p, dt=d.BF16_F32: lib.gemm_run_dact(  # noqa: E731
        h, 0, 0, M, N, K, 1.0, p, K, p, N, act, kind, z, ldz, s, lds, None, C, N, dt)
    assert dact(h=None) == 3
    for kw in (dict(act=9), dict(kind=0), dict(kind=4), dict(z=None), dict(ldz=N - 1), dict(kind=2), dict(C=None),
               dict(kind=2, s=p, lds=1), dict(dt=d.E4M3_E4M3)):
        assert dact(**kw) == 1, kw
    mx = lambda h=h, r=8, c=64, act=1, z=p, ldz=64, o=p, q=p, s=p, lds=2: lib.gemm_act_mx(  # noqa: E731
        h, r, c, act, z, ldz, o, 64, q, 64, s, lds)
    assert mx(h=None) == 3
    for kw in (dict(r=-1), dict(c=-1), dict(act=7), dict(z=None), dict(o=None), dict(q=None), dict(s=None), dict(ldz=63),
               dict(lds=1)):
        assert mx(**kw) == 1, kw
    assert mx(r=0, z=None) == 0
    g = lambda h=h, r=8, act=1, q=p, s=p, lds=2, dh=p, dz=p, db=p, o=p, ldo=64: lib.gemm_act_grad_mx(  # noqa: E731
        h, r, 64, act, q, 64, s, lds, dh, 64, dz, 64, db, o, ldo)
    assert g(h=None) == 3
    for kw in (dict(r=-1), dict(act=7), dict(q=None), dict(s=None), dict(lds=1), dict(dh=None), dict(dz=None, db=None),
               dict(dh=None, dz=None, db=None, o=None), dict(ldo=63)):
        assert g(**kw) == 1, kw
    ln = lambda h=h, r=8, c=64, x=p, ldx=64, xt=1, g=p, wt=1, eps=1e-5, y=p, yt=1: lib.gemm_layernorm(  # noqa: E731
        h, r, c, x, ldx, xt, g, None, wt, eps, y, 64, yt, None, None)
    assert ln(h=None) == 3
    for kw in (dict(r=-1), dict(c=-2), dict(x=None), dict(y=None), dict(ldx=63), dict(xt=2), dict(yt=-1), dict(wt=2)):
        assert ln(**kw) == 1, kw
    assert ln(eps=-1.0) == 2 and ln(eps=float("nan")) == 2 and ln(eps=float("inf")) == 2
    lg = lambda h=h, r=8, dy=p, x=p, mu=p, rs=p, g=p, wt=1, dr=p, ldr=64, dx=p, yt=1: lib.gemm_layernorm_grad(  # noqa: E731
        h, r, 64, dy, 64, yt, x, 64, 1, mu, rs, g, wt, dr, ldr, dx, 64, p, p)
    assert lg(h=None) == 3
    for kw in (dict(r=-1), dict(dy=None), dict(x=None), dict(mu=None), dict(rs=None), dict(dx=None), dict(wt=2),
               dict(ldr=63), dict(yt=2)):
        assert lg(**kw) == 1, kw
    torch.cuda.synchronize()
    assert (buf == 7).all()


def test_refusals_of_the_binding(gpu):
    import torch
    cu = dict(device="cuda")
    A, B, C = (torch.zeros(32, 32, dtype=torch.bfloat16, **cu) for _ in range(3))
    q, s = torch.zeros(32, 32, dtype=torch.uint8, **cu), torch.zeros(32, 1, dtype=torch.uint8, **cu)
    v = torch.zeros(32, **cu)
    bad = [
        lambda: gpu.run_act(A, B, C, act="tanh"),
        lambda: gpu.run_act(A, B[:16], C),
        lambda: gpu.run_act(A, B, C[:, :16]),
        lambda: gpu.run_act(A, B.float(), C),
        lambda: gpu.run_act(A, B, C.half()),
        lambda: gpu.run_act(A, B, C, bias=v[:16]),
        lambda: gpu.run_act(A, B, C, bias=v.double()),
        lambda: gpu.run_act(A, B, C, residual=C.float()),
        lambda: gpu.run_act(A, B, C, z=q),
        lambda: gpu.run_act(A, B, C, z=q, z_scales=s[:16]),
        lambda: gpu.run_act(A, B, C, z=C[:16]),
        lambda: gpu.run_act(A.cpu(), B, C),
        lambda: gpu.run_dact(A, B, C, q),
        lambda: gpu.run_dact(A, B, C, C, dbias=v.bfloat16()),
        lambda: gpu.act_mx(A.float(), C, q, s),
        lambda: gpu.act_mx(A, C, q, None),
        lambda: gpu.act_grad_mx(q, s, act="relu", dh=A.float(), dz=C),
        lambda: gpu.layernorm(A, C.half()),
        lambda: gpu.layernorm(A, C, gamma=v, beta=v.bfloat16()),
        lambda: gpu.layernorm(A, C, mean=v[:5]),
        lambda: gpu.layernorm_grad(A, A, v, v, C.float()),
        lambda: gpu.layernorm_grad(A, A, v, v, C, dgamma=v.cpu()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(i)
