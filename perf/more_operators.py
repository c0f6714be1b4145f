"""The gated feed-forward operators that are measured, and their plain forms.

Five calls: both projections of a gated block with the activation and the product of the two behind
them (run_gated), the product that runs back through it (run_dgated), rows quantised to 8-bit integers
with a scale each (quantize_i8), the product of such codes with a scale for each token and channel
(run_i8) and its gated form (run_gated_i8).  `own` chooses between the framework's calls and the plain
forms: elementary torch operations in 32 bits, rounded once at the end.

The 8-bit format: a row's scale is its largest magnitude over 127, its codes are the whole numbers
nearest to 127 x / (largest magnitude), ties to even.
"""
import functools
import math

import torch

own = False

DEVICE = "cuda:0"
ACTS = ("relu", "gelu", "gelu_tanh", "silu")
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1, "i8": 1}
GATED = ("run_gated", "run_gated_i8")
LARGEST = 2 * 8192 * 13696 * 5120  # multiply-adds of the largest listed case


# ------------------------------------------------------------------------------------- cases
# 13696 = 8/3 5120 and 10944 = 8/3 4096, rounded up to whole tiles: the hidden width at which a gated
# block has the parameters of a plain one of 4 times the model's width.

def listed():
    return [
        # one token through both projections in the serving loop: the weights are read once
        dict(name="gated_decode_1", op="run_gated", m=1, n=10944, k=4096, dtype="bf16", out="bf16", layout="nt",
             act="silu", bias=False, keep=False),
        # a ragged micro-batch with biases and weights as [in][out], both arguments kept for the backward pass
        dict(name="gated_ragged", op="run_gated", m=1531, n=2736, k=1000, dtype="bf16", out="f32", layout="nn",
             act="gelu", bias=True, keep=True),
        # a training step: both arguments kept
        dict(name="gated_train", op="run_gated", m=4096, n=13696, k=5120, dtype="bf16", out="bf16", layout="nt",
             act="silu", bias=False, keep=True),
        # E4M3 prefill of a long prompt
        dict(name="gated_prefill_e4m3", op="run_gated", m=8192, n=13696, k=5120, dtype="e4m3", out="bf16", layout="nt",
             act="silu", bias=False, keep=False),
        # backward through the down-projection and the gate on a ragged micro-batch, with bias gradients
        dict(name="dgated_ragged", op="run_dgated", m=1531, n=2736, k=1000, dtype="bf16", out="f32", layout="nt",
             act="gelu_tanh", sums=True, restore=False),
        # the same in a training step, the hidden activation computed again for the weight gradient behind it
        dict(name="dgated_train", op="run_dgated", m=4096, n=13696, k=5120, dtype="bf16", out="bf16", layout="nn",
             act="silu", sums=False, restore=True),
        # the tokens of a decoding batch, in front of an integer product
        dict(name="quantize_decode_24", op="quantize_i8", m=24, n=13696, x="bf16"),
        # the tokens of a long prompt
        dict(name="quantize_prefill", op="quantize_i8", m=16384, n=5120, x="bf16"),
        # down-projection of a few tokens onto the residual stream, weights as [in][out]
        dict(name="i8_decode_5", op="run_i8", m=5, n=5120, k=13696, out="bf16", layout="nn", act="none", bias=False,
             residual=True),
        # down-projection of a long prompt onto the residual stream
        dict(name="i8_prefill", op="run_i8", m=8192, n=5120, k=13696, out="bf16", layout="nt", act="none", bias=True,
             residual=True),
        # both projections for a decoding batch
        dict(name="gated_i8_decode_24", op="run_gated_i8", m=24, n=13696, k=5120, out="bf16", layout="nt", act="silu",
             bias=False),
        # both projections of a long prompt
        dict(name="gated_i8_prefill", op="run_gated_i8", m=8192, n=13696, k=5120, out="bf16", layout="nt", act="silu",
             bias=False),
    ]


def _spread(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["run_gated", "run_gated", "run_dgated", "quantize_i8", "run_i8", "run_gated_i8"])
    if op == "quantize_i8":
        n = _spread(rng, 64, 20480)
        return dict(op=op, m=_spread(rng, 1, max(1, min(65536, 16384 * 5120 // n))), n=n, x=rng.choice(["bf16", "f32"]))
    # tokens: any number; features: multiples of 16, as weights have them
    m = _spread(rng, 64, 8192) if op == "run_dgated" else _spread(rng, 1, 16384)
    n, k = (_spread(rng, 256, 20480) // 16 * 16 for _ in range(2))
    while m * n * k * (2 if op in GATED else 1) > LARGEST // 2:
        n, k = max(256, n // 32 * 16), max(256, k // 32 * 16)
    case = dict(op=op, m=m, n=n, k=k, layout=rng.choice(["nt", "nn"]), out=rng.choice(["bf16", "bf16", "f32"]),
                act=rng.choice(ACTS))
    if op == "run_gated":
        return dict(case, dtype=rng.choice(["bf16", "bf16", "e4m3"]), bias=rng.random() < 0.3, keep=rng.random() < 0.5)
    if op == "run_dgated":
        return dict(case, dtype="bf16", sums=rng.random() < 0.3, restore=rng.random() < 0.5)
    if op == "run_i8":
        return dict(case, act=rng.choice(("none",) + ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5)
    return dict(case, bias=rng.random() < 0.3)


# ------------------------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)

    def normal(*shape, std=1.0, dtype="f32"):
        v = torch.randn(shape, generator=g, device=DEVICE).mul_(std)
        return v.clamp_(-448.0, 448.0).to(DTYPES[dtype]) if dtype == "e4m3" else v.to(DTYPES[dtype])

    def empty(*shape, dtype="f32"):
        return torch.empty(shape, device=DEVICE, dtype=DTYPES[dtype])

    def tokens(m, n):
        # rows of unlike spreads, a few channels larger than the others, as activations have them
        x = torch.randn((m, n), generator=g, device=DEVICE)
        x.mul_(torch.rand((m, 1), generator=g, device=DEVICE).mul_(1.5).add_(0.5))
        return x.mul_(torch.where(torch.rand((1, n), generator=g, device=DEVICE) < 0.004, 12.0, 1.0))

    s, op, m, n = dict(case), case["op"], case["m"], case["n"]
    if op == "quantize_i8":
        s["X"] = tokens(m, n).to(DTYPES[case["x"]])
        s["Q"], s["S"] = empty(m, n, dtype="i8"), empty(m)
        return s
    k = case["k"]
    shape = (n, k) if case["layout"] == "nt" else (k, n)
    if op in ("run_i8", "run_gated_i8"):
        s["A"], s["SA"] = _quantize(tokens(m, k))
        for b in ("B", "B2")[:2 if op in GATED else 1]:
            # a scale for each output channel
            w, s["S" + b] = _quantize(normal(n, k, std=k ** -0.5))
            s[b] = w if case["layout"] == "nt" else w.t().contiguous()
    else:
        dt = case["dtype"]
        # weights that keep the variance (E4M3: at unit scale, alpha carries it)
        std = 1.0 if dt == "e4m3" else k ** -0.5
        s["alpha"] = k ** -0.5 if dt == "e4m3" else 1.0
        s["A"] = normal(m, k, dtype=dt)
        for b in ("B", "B2")[:2 if op in GATED else 1]:
            s[b] = normal(*shape, std=std, dtype=dt)
    s["C"] = empty(m, n, dtype=case["out"])
    if op == "run_dgated":
        s["G"], s["U"] = normal(m, n, dtype="bf16"), normal(m, n, dtype="bf16")
        s["dU"] = empty(m, n, dtype=case["out"])
        s["H"] = empty(m, n, dtype="bf16") if case["restore"] else None
        s["sg"], s["su"] = (empty(n), empty(n)) if case["sums"] else (None, None)
    else:
        s["b"] = normal(n, std=0.1) if case["bias"] else None
        s["b2"] = normal(n, std=0.1) if case["bias"] and op in GATED else None
        s["R"] = normal(m, n, dtype=case["out"]) if case.get("residual") else None
        s["G"], s["U"] = (empty(m, n, dtype="bf16"), empty(m, n, dtype="bf16")) if case.get("keep") else (None, None)
    return s


# --------------------------------------------------------------------------------- plain forms

def _quantize(x):
    """Rows -> (codes, scales).  The quotients in 64 bits: a value next to the middle between two codes
    would fall on the wrong side in 32."""
    x = x.float()
    top = x.abs().amax(1, keepdim=True)
    q = torch.round(x.double() * 127.0 / top.double())
    return torch.where(top > 0, q, torch.zeros_like(q)).to(torch.int8), top[:, 0] / 127.0


def _logistic(v):
    return 1.0 / (1.0 + torch.exp(-v))


_C0, _C1 = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return z * _logistic(2.0 * _C0 * (z + _C1 * z * z * z))
    if act == "silu":
        return z * _logistic(z)
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        phi = torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * phi
    if act == "gelu_tanh":
        s = _logistic(2.0 * _C0 * (z + _C1 * z * z * z))
        return s + z * s * (1.0 - s) * 2.0 * _C0 * (1.0 + 3.0 * _C1 * z * z)
    s = _logistic(z)
    return s * (1.0 + z * (1.0 - s))


def _product(s, b="B"):
    w = s[b].float()
    p = s["A"].float() @ (w.t() if s["layout"] == "nt" else w)
    p = p * s["SA"][:, None] * s["S" + b] if "SA" in s else p * s["alpha"]
    bias = s.get("b" + b[1:])
    return p if bias is None else p + bias


def _plain(s):
    op = s["op"]
    if op == "quantize_i8":
        q, scales = _quantize(s["X"])
        return {"Q": q, "S": scales}
    if op == "run_i8":
        c = _act(_product(s), s["act"])
        return {"C": (c if s["R"] is None else c + s["R"].float()).to(s["C"].dtype)}
    if op in GATED:
        z, u = _product(s), _product(s, "B2")
        out = {"C": (_act(z, s["act"]) * u).to(s["C"].dtype)}
        if s["G"] is not None:
            out["G"], out["U"] = z.to(torch.bfloat16), u.to(torch.bfloat16)
        return out
    d, z, u = _product(s), s["G"].float(), s["U"].float()
    h = _act(z, s["act"])
    dg, du = d * u * _act_slope(z, s["act"]), d * h
    out = {"dG": dg.to(s["C"].dtype), "dU": du.to(s["dU"].dtype)}
    if s["sg"] is not None:
        out["sg"], out["su"] = dg.sum(0), du.sum(0)
    if s["H"] is not None:
        out["H"] = (h * u).to(torch.bfloat16)
    return out


# ------------------------------------------------------------------------- the framework's calls

@functools.lru_cache(maxsize=None)
def _handle():
    import dense_blas3_gemm_amd as d
    return d.Gemm(0)


def _framework(s):
    h, op = _handle(), s["op"]
    if op == "quantize_i8":
        h.quantize_i8(s["X"], s["Q"], s["S"])
        return {"Q": s["Q"], "S": s["S"]}
    nt = s["layout"] == "nt"
    if op == "run_i8":
        h.run_i8(s["A"], s["SA"], s["B"], s["SB"], s["C"], transB=nt, act=s["act"], bias=s["b"], residual=s["R"])
        return {"C": s["C"]}
    if op == "run_gated_i8":
        h.run_gated_i8(s["A"], s["SA"], s["B"], s["SB"], s["B2"], s["SB2"], s["C"], transB=nt, act=s["act"],
                       bias_g=s["b"], bias_u=s["b2"])
        return {"C": s["C"]}
    if op == "run_gated":
        h.run_gated(s["A"], s["B"], s["B2"], s["C"], transB=nt, alpha=s["alpha"], act=s["act"], bias_g=s["b"],
                    bias_u=s["b2"], g=s["G"], u=s["U"])
        return {"C": s["C"], **({} if s["G"] is None else {"G": s["G"], "U": s["U"]})}
    h.run_dgated(s["A"], s["B"], s["G"], s["U"], s["C"], s["dU"], transB=nt, alpha=s["alpha"], act=s["act"], h=s["H"],
                 dbias_g=s["sg"], dbias_u=s["su"])
    out = {"dG": s["C"], "dU": s["dU"]}
    if s["sg"] is not None:
        out["sg"], out["su"] = s["sg"], s["su"]
    if s["H"] is not None:
        out["H"] = s["H"]
    return out


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------- work

def work(case):
    op, m, n = case["op"], case["m"], case["n"]
    if op == "quantize_i8":
        return {"bytes": m * n * (BYTES[case["x"]] + 1) + 4 * m, "flops": 3 * m * n}
    k, o, b = case["k"], BYTES[case["out"]], 2 if op in GATED else 1
    e = BYTES[case.get("dtype", "i8")]
    moved = (m * k + b * n * k) * e + m * n * o + 4 * b * n * case.get("bias", False)
    if op.endswith("i8"):
        moved += 4 * (m + b * n) + m * n * o * case.get("residual", False)
    elif op == "run_gated":
        moved += 4 * m * n * case["keep"]
    else:
        moved += m * n * (4 + o + 2 * case["restore"]) + 8 * n * case["sums"]
    return {"bytes": moved, "flops": 2 * b * m * n * k}


# ------------------------------------------------------------------------------- 64-bit results

def _exact_act(z, act):
    """(act(z), act'(z)) in 64 bits, from tanh and erfc."""
    one = torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0.0), torch.heaviside(z, torch.zeros_like(z))
    if act == "gelu":
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
        return z * p, p + z * torch.exp(-z.square() / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_C0 * (z + _C1 * z.pow(3)))
        return 0.5 * z * (one + t), 0.5 * (one + t) + 0.5 * z * (one - t.square()) * _C0 * (one + 3.0 * _C1 * z.square())
    if act == "silu":
        s = 0.5 * (one + torch.tanh(0.5 * z))
        return z * s, s + z * s * (one - s)
    return z, one


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    up = lambda t: t.double()  # noqa: E731
    if op == "quantize_i8":
        x = up(s["X"])
        scale = torch.maximum(x.max(1).values, -x.min(1).values) / 127.0
        return {"Q": None, "S": scale}

    def product(b, scales, bias):
        w = up(s[b])
        p = torch.mm(up(s["A"]), w.T if case["layout"] == "nt" else w)
        if op.endswith("i8"):
            p.mul_(torch.outer(up(s["SA"]), up(s[scales])))
        else:
            p.mul_(s["alpha"])
        return p if s.get(bias) is None else p.add_(up(s[bias]))

    p = product("B", "SB", "b")
    if op == "run_i8":
        c = _exact_act(p, case["act"])[0]
        return {"C": c + up(s["R"]) if case["residual"] else c}
    if op in GATED:
        v = product("B2", "SB2", "b2")
        out = {"C": _exact_act(p, case["act"])[0] * v}
        return {**out, "G": p, "U": v} if case.get("keep") else out
    z, u = up(s["G"]), up(s["U"])
    a, slope = _exact_act(z, case["act"])
    out = {"dU": p * a, "dG": p * slope * u}
    if case["sums"]:
        out["sg"], out["su"] = out["dG"].sum(0), out["dU"].sum(0)
    if case["restore"]:
        out["H"] = a * u
    return out
