"""The MLP-block operators where their row loops go round: many rows to a thread or a workgroup,
products in more than one block of rows, column sums over many partial rows.

Where it can be had the check is exact: small whole numbers, whose products and sums fp32 holds
(below 2^24), so that a lost, doubled or misplaced row is a wrong number and no rounding hides it.
The other bounds are those of test_gpu_mlp.py, against torch in float64.
"""
import pytest

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EVAL = 1e-6
EPS = 1e-3
DT = {"bf16": 2.0 ** -8, "f32": 2.0 ** -22}


def types():
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}


def ints(gen, lo, hi, *shape, kind="f32", pad=0):
    """Whole numbers lo .. hi in rows of shape[-1] + pad elements."""
    import torch
    whole = torch.randint(lo, hi + 1, (*shape[:-1], shape[-1] + pad), generator=gen, device="cuda").to(types()[kind])
    return whole[..., :shape[-1]]


def within(got, want, bound, what):
    bad = ~((got - want).abs() <= bound)
    assert not bad.any().item(), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {((got - want).abs() / bound).max().item():.3g} of its bound"


# ---------------------------------------------------------------------------------- layer norm
# Rounds of a workgroup at these shapes, bf16 (forward / gradient; past 16384 columns also the rows to a
# thread of the weights' sums): 1531 x 4099 2 / 3, 3000 x 1100 2 / 2, 100000 x 72 2 / 4, 1100 x 8200 5 / 5,
# 5003 x 5120 7 / 10, 700 x 17515 3 / 3 and 4 rows, 600 x 40001 1 / 1 and 6 rows.  fp32 gradients make
# up to twice as many.
NORMS = [(1531, 4099), (3000, 1100), (100000, 72), (1100, 8200), (5003, 5120), (700, 17515), (600, 40001)]
KINDS = [("bf16", "bf16", "f32"), ("f32", "bf16", "bf16"), ("f32", "f32", None), ("bf16", "f32", "f32")]


def chain(N):
    return -(-N // 64) + 16


@pytest.mark.parametrize("shape", NORMS)
@pytest.mark.parametrize("kinds", KINDS)
def test_layernorm_rounds(gpu, shape, kinds):
    import torch
    (M, N), (xk, yk, wk) = shape, kinds
    gen = torch.Generator(device="cuda").manual_seed(N + KINDS.index(kinds))
    f = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = (f(M, N) * (0.5 + 1.5 * torch.rand(M, 1, generator=gen, device="cuda")) + 2 * f(M, 1)).to(types()[xk])
    g = (1 + 0.2 * f(N)).to(types()[wk]) if wk else None
    b = f(N).to(types()[wk]) if wk else None
    y = torch.full((M, N + 3), -77.0, dtype=types()[yk], device="cuda")
    mean, rstd = (torch.full((M,), float("nan"), device="cuda") for _ in range(2))
    gpu.layernorm(x, y[:, :N], gamma=g, beta=b, eps=EPS, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    assert (y[:, N:] == -77.0).all()
    xv = x.double()
    mu = xv.mean(1, keepdim=True)
    r = 1 / torch.sqrt((xv - mu).square().mean(1, keepdim=True) + EPS)
    n = (xv - mu) * r
    want = n if g is None else n * g.double() + b.double()
    d = chain(N)
    e_mu = d * U * xv.abs().mean(1, keepdim=True)
    e_r = r * (0.5 * (d + 6) * U + r * r * e_mu * ((xv - mu).abs().mean(1, keepdim=True) + e_mu) + 4 * U)
    within(mean.double()[:, None], mu, e_mu, "mean")
    within(rstd.double()[:, None], r, e_r, "rstd")
    ga, ba = (g.double().abs(), b.double().abs()) if wk else (1.0, 0.0)
    err = ga * ((e_mu + 2 * U * xv.abs()) * r + (xv - mu).abs() * (e_r + 2 * U * r)) + 2 * U * (want.abs() + ba)
    within(y[:, :N].double(), want, err + DT[yk] * want.abs(), "y")


# (one type each of the single sums)
@pytest.mark.parametrize("shape,kinds,sums",
                         [(s, k, w) for i, s in enumerate(NORMS) for j, k in enumerate(KINDS)
                          for w in ("both", "none") + (("dgamma", "dbeta") if j == i % 4 else ())])
def test_layernorm_grad_rounds(gpu, shape, kinds, sums):
    """Whole numbers with mean 0 and rstd 1: the weights' sums are exact."""
    import torch
    (M, N), (xk, yk, wk) = shape, kinds
    gen = torch.Generator(device="cuda").manual_seed(N)
    x, dy = ints(gen, -8, 8, M, N, kind=xk), ints(gen, -4, 4, M, N, kind=yk)
    res = ints(gen, -9, 9, M, N, kind=xk) if KINDS.index(kinds) % 2 else None
    g = ints(gen, 1, 3, N, kind=wk) if wk else None
    mean, rstd = torch.zeros(M, device="cuda"), torch.ones(M, device="cuda")
    dx = torch.full((M, N + 3), -77.0, dtype=types()[xk], device="cuda")
    dg, db = (torch.full((N,), float("nan"), device="cuda") for _ in range(2))
    gpu.layernorm_grad(dy, x, mean, rstd, dx[:, :N], gamma=g, dgamma=dg if sums in ("both", "dgamma") else None,
                       dbeta=db if sums in ("both", "dbeta") else None, residual=res)
    torch.cuda.synchronize()
    assert (dx[:, N:] == -77.0).all()
    xv, dv = x.double(), dy.double()
    if sums in ("both", "dgamma"):
        assert torch.equal(dg.double(), (dv * xv).sum(0))
    if sums in ("both", "dbeta"):
        assert torch.equal(db.double(), dv.sum(0))
    gv = dv if g is None else dv * g.double()
    c1, c2 = gv.mean(1, keepdim=True), (gv * xv).mean(1, keepdim=True)
    want = gv - c1 - xv * c2 + (0 if res is None else res.double())
    # the row sums are exact too: their division, and the roundings of the combination
    err = 4 * U * (gv.abs() + c1.abs() + 2 * xv.abs() * c2.abs() + want.abs())
    within(dx[:, :N].double(), want, err + DT[xk] * want.abs() + 1e-30, "dx")


# ------------------------------------------------------------- 8-bit checkpoints of activations
# Rows to a thread (act_mx / act_grad_mx with bias sums, four at a time): 2047 x 5000 and 5003 2 / 8, 9001 x
# 1000 2 / 5, 5001 x 2049 3 / 8, 100001 x 96 and 100003 x 93 2 / 5, 8195 x 20480 21 / 41.
ROWS = [(2047, 5000), (2047, 5003), (9001, 1000), (5001, 2049), (100001, 96), (100003, 93), (8195, 20480)]


def block_values(q, s):
    import torch
    f = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), s.int() - 127)
    return q.view(torch.float8_e4m3fn).double() * f.repeat_interleave(32, 1)[:, :q.shape[1]]


def mx_buffers(M, N):
    import torch
    return (torch.full((M, N), 0x5A, dtype=torch.uint8, device="cuda"),
            torch.full((M, (N + 31) // 32), 0x5A, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("shape", ROWS)
def test_act_mx_rows(gpu, shape):
    import torch
    M, N = shape
    gen = torch.Generator(device="cuda").manual_seed(M)
    z = torch.randn(M, N, generator=gen, device="cuda").bfloat16()
    want_q, want_s = mx_buffers(M, N)
    gpu.quantize_mx(z, want_q, want_s)
    for act in ("relu", "silu"):
        q, s = mx_buffers(M, N)
        h = torch.full((M, N + 1), -77.0, dtype=torch.bfloat16, device="cuda")
        gpu.act_mx(z, h[:, :N], q, s, act=act)
        torch.cuda.synchronize()
        assert torch.equal(q, want_q) and torch.equal(s, want_s) and (h[:, N:] == -77.0).all()
        if act == "relu":
            assert torch.equal(h[:, :N], z.clamp(min=0))
        else:
            for m in range(0, M, 16384):
                zv = z[m:m + 16384].double()
                want = zv * torch.sigmoid(zv)
                within(h[m:m + 16384, :N].double(), want, DT["bf16"] * want.abs() + EVAL * zv.abs() + 1e-38, act)


@pytest.mark.parametrize("shape", ROWS)
def test_act_grad_mx_rows(gpu, shape):
    """Whole numbers: the sums are exact, and so is what the codes hold (15 becomes 14 in a block without
    a 16: past the format's largest value)."""
    import torch
    M, N = shape
    gen = torch.Generator(device="cuda").manual_seed(M + 1)
    z, dh = ints(gen, -16, 16, M, N, kind="bf16"), ints(gen, -8, 8, M, N, kind="bf16", pad=1)
    q, s = mx_buffers(M, N)
    gpu.quantize_mx(z, q, s)
    z = torch.cat([block_values(q[m:m + 16384], s[m:m + 16384]).bfloat16() for m in range(0, M, 16384)])
    on = z > 0
    want = torch.where(on, dh, torch.zeros_like(dh))
    for act, D, H in (("relu", want, torch.where(on, z, torch.zeros_like(z))), ("none", dh, z)):
        for with_dz, with_db, with_h in ((1, 1, 1), (0, 1, 0), (1, 0, 1)):
            dz = torch.full((M, N + 1), -77.0, dtype=torch.bfloat16, device="cuda") if with_dz else None
            h = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda") if with_h else None
            db = torch.full((N,), float("nan"), device="cuda") if with_db else None
            gpu.act_grad_mx(q, s, act=act, dh=dh, dz=dz[:, :N] if with_dz else None, dbias=db, h=h)
            torch.cuda.synchronize()
            if with_dz:
                assert torch.equal(dz[:, :N], D) and (dz[:, N:] == -77.0).all(), act
            if with_h:
                assert torch.equal(h, H), act
            if with_db:
                assert torch.equal(db, D.double().sum(0).float()), act
    # a slope of its own for every element
    dz = torch.empty_like(z)
    z = torch.randn(M, N, generator=gen, device="cuda").bfloat16()
    gpu.quantize_mx(z, q, s)
    gpu.act_grad_mx(q, s, act="silu", dh=dh, dz=dz)
    torch.cuda.synchronize()
    for m in range(0, M, 16384):
        zv, dv = block_values(q[m:m + 16384], s[m:m + 16384]), dh[m:m + 16384].double()
        sg = torch.sigmoid(zv)
        w = dv * sg * (1 + zv * (1 - sg))
        within(dz[m:m + 16384].double(), w, DT["bf16"] * w.abs() + EVAL * dv.abs() * (1 + zv.abs()) + 1e-38, "silu")


# ------------------------------------------------------------------------------------- products
# N no multiple of 8, or operands at odd addresses: an fp32 product in the workspace, 192 MiB of it
# at a time (50.3 million values), and the epilogue over each block of rows.  Two blocks: 69376 rows
# of 723 columns (rows of 724) and the rest; 17152 of 2931, twice, and the rest.
BLOCKS = [(70001, 723, 16, (0, 0)), (70001, 723, 16, (0, 1)), (70008, 723, 16, (1, 1)), (70001, 723, 16, (1, 0)),
          (35000, 2931, 24, (0, 1))]


def operands(gen, M, N, K, trans, kind="bf16"):
    A = ints(gen, -2, 2, *((K, M) if trans[0] else (M, K)), kind=kind)
    B = ints(gen, -2, 2, *((N, K) if trans[1] else (K, N)), kind=kind)
    P = (A.t() if trans[0] else A).float() @ (B.t() if trans[1] else B).float()
    return A, B, P


def without_zero_signs(q):
    return q * ((q & 0x7F) != 0)


@pytest.mark.parametrize("case", BLOCKS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_run_act_blocks_of_rows(gpu, case, out):
    import torch
    M, N, K, trans = case
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    A, B, P = operands(gen, M, N, K, trans)
    bias = ints(gen, -3, 3, N)
    R = ints(gen, -5, 5, M, N, kind=out, pad=1)
    Z = P + bias
    want = Z.clamp(min=0) + 2 * R.float()
    C = torch.full((M, N + 2), -77.0, dtype=types()[out], device="cuda")
    q, s = mx_buffers(M, N)
    gpu.run_act(A, B, C[:, :N], transA=trans[0], transB=trans[1], act="relu", bias=bias, residual=R, beta=2.0, z=q,
                z_scales=s)
    want_q, want_s = mx_buffers(M, N)
    gpu.quantize_mx(Z.bfloat16(), want_q, want_s)  # (|Z| < 256)
    torch.cuda.synchronize()
    assert torch.equal(C[:, :N].float(), want) and (C[:, N:] == -77.0).all()
    assert torch.equal(s, want_s) and torch.equal(without_zero_signs(q), without_zero_signs(want_q))
    zb = torch.full((M, N + 1), -77.0, dtype=torch.bfloat16, device="cuda")
    C.fill_(-77.0)
    C[:, :N] = R
    gpu.run_act(A, B, C[:, :N], transA=trans[0], transB=trans[1], act="none", bias=bias, residual=C[:, :N], z=zb[:, :N])
    torch.cuda.synchronize()
    assert torch.equal(C[:, :N].float(), Z + R.float()) and torch.equal(zb[:, :N].float(), Z)
    assert (C[:, N:] == -77.0).all() and (zb[:, N:] == -77.0).all()


@pytest.mark.parametrize("case", BLOCKS)
@pytest.mark.parametrize("z_kind", ["bf16", "mx"])
def test_run_dact_blocks_of_rows(gpu, case, z_kind):
    import torch
    M, N, K, trans = case
    gen = torch.Generator(device="cuda").manual_seed(M - N)
    A, B, P = operands(gen, M, N, K, trans)
    z = ints(gen, -2, 2, M, N, kind="bf16", pad=1)
    want = torch.where(z > 0, P, torch.zeros_like(P))
    scales = None
    if z_kind == "mx":
        q, scales = mx_buffers(M, N)
        gpu.quantize_mx(z, q, scales)
        z = q
    C = torch.full((M, N + 2), -77.0, device="cuda")
    db = torch.full((N,), float("nan"), device="cuda")
    gpu.run_dact(A, B, C[:, :N], z, z_scales=scales, transA=trans[0], transB=trans[1], act="relu", dbias=db)
    torch.cuda.synchronize()
    assert torch.equal(C[:, :N], want) and (C[:, N:] == -77.0).all()
    assert torch.equal(db, want.double().sum(0).float())


# every way of a product with bias sums: a few rows, ring tiles unsplit and split, 256 x 256 tiles,
# two launches cut by columns and by rows
@pytest.mark.parametrize("shape", [(13, 512, 256), (64, 264, 512), (40, 136, 8192), (300, 520, 256), (1000, 2056, 520),
                                   (4096, 4096, 128), (1300, 13088, 320), (13104, 1296, 320), (30001, 256, 64),
                                   (4099, 17, 40)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_run_dact_sums_are_exact(gpu, shape, kind):
    import torch
    M, N, K = shape
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    A, B, P = operands(gen, M, N, K, (0, 1))
    if kind == "e4m3":
        A, B = A.to(torch.float8_e4m3fn), B.to(torch.float8_e4m3fn)
    z = ints(gen, -2, 2, M, N, kind="bf16")
    want = torch.where(z > 0, P, torch.zeros_like(P))
    C, db = torch.empty(M, N, device="cuda"), torch.full((N,), float("nan"), device="cuda")
    gpu.run_dact(A, B, C, z, transB=1, act="relu", dbias=db)
    torch.cuda.synchronize()
    assert torch.equal(C, want)
    assert torch.equal(db, want.double().sum(0).float())


# The partial rows of the bias sums of a fused product have the workspace past its first 64 MiB; where
# they do not fit there, the product goes by blocks of rows.  With a partial row to 64 or 128 rows
# (tiles of 128 or 256 rows) 29696 x 98304 fits and 73728 x 98304 does not.
@pytest.mark.parametrize("shape", [(29696, 98304), (73728, 98304)])
def test_run_dact_sums_of_the_largest(gpu, shape):
    import torch
    (M, N), K = shape, 8
    gen = torch.Generator(device="cuda").manual_seed(M)
    A, B = ints(gen, -2, 2, M, K, kind="bf16"), ints(gen, -2, 2, N, K, kind="bf16")
    z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    sums = torch.zeros(N, dtype=torch.float64, device="cuda")
    for m in range(0, M, 2048):
        z[m:m + 2048] = ints(gen, -2, 2, min(2048, M - m), N, kind="bf16")
    C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    db = torch.full((N,), float("nan"), device="cuda")
    gpu.run_dact(A, B, C, z, transB=1, act="relu", dbias=db)
    torch.cuda.synchronize()
    for m in range(0, M, 2048):
        want = torch.where(z[m:m + 2048] > 0, A[m:m + 2048].float() @ B.t().float(), 0.0)
        assert torch.equal(C[m:m + 2048].float(), want), m  # (|D| <= 32)
        sums += want.double().sum(0)
    assert torch.equal(db, sums.float())
    del z, C
    torch.cuda.empty_cache()


def test_epilogue_tiles_serve_no_plain_product(gpu):
    import torch
    import dense_blas3_gemm_amd as d
    names = [n for n in d.policies() if n.startswith("ep_")]
    assert names
    A, B = (torch.ones(256, 256, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    C = torch.full((256, 256), -77.0, dtype=torch.bfloat16, device="cuda")
    for n in names:
        gpu.set_policy(n)
        try:
            with pytest.raises(d.GemmError) as e:
                gpu(A, B, C)
        finally:
            gpu.set_policy(None)
        assert e.value.status == 2, n
    torch.cuda.synchronize()
    assert (C == -77).all()


# a few rows, ring tiles unsplit and split, 256 x 256 tiles, two launches, blocks of rows
@pytest.mark.parametrize("shape", [(13, 512, 1000), (300, 520, 256), (40, 136, 8192), (2048, 1536, 520), (1300, 13088, 320),
                                   (130, 99, 264)])
def test_codes_are_those_of_the_fp32_argument(gpu, shape):
    """The codes and scales that a product leaves are its fp32 Z's, bit for bit (some two dozen rows)."""
    import numpy as np
    import oracle
    import torch
    M, N, K = shape
    gen = torch.Generator(device="cuda").manual_seed(K)
    A, B = (torch.randn(n, K, generator=gen, device="cuda").bfloat16() for n in (M, N))
    b = torch.randn(N, generator=gen, device="cuda")
    Z, C = torch.empty(M, N, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    q, s = mx_buffers(M, N)
    gpu.run_act(A, B, Z, transB=1, alpha=0.1, act="none", bias=b)
    gpu.run_act(A, B, C, transB=1, alpha=0.1, act="gelu_tanh", bias=b, z=q, z_scales=s)
    torch.cuda.synchronize()
    some = slice(0, M, max(1, M // 24))
    codes, scales = oracle.quantize_mx(Z[some].cpu().numpy().astype(np.float64))
    assert np.array_equal(s[some].cpu().numpy(), scales) and np.array_equal(q[some].cpu().numpy(), codes)
