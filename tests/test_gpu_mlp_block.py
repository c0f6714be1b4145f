"""The operators together, as examples/mlp_block.py uses them, against the same block in float64
autograd on the values the operators are given."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

ACTS = {"gelu_tanh": lambda t: t * 0.5 * (1 + (0.7978845608028654 * (t + 0.044715 * t ** 3)).tanh()),
        "silu": lambda t: t / (1 + (-t).exp()), "relu": lambda t: t.clamp(min=0)}


def block64(b, x, act):
    """y and the tensors to differentiate, in float64 on the CPU"""
    import torch
    p = {k: getattr(b, k).detach().double().cpu().requires_grad_(True) for k in ("gamma", "beta", "w1", "b1", "w2", "b2")}
    x = x.double().cpu().requires_grad_(True)
    mean = x.mean(1, keepdim=True)
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    n = (x - mean) / torch.sqrt(var + 1e-5) * p["gamma"] + p["beta"]
    z = n @ p["w1"].T + p["b1"]
    return ACTS[act](z) @ p["w2"].T + p["b2"] + x, x, p


def rel(got, want):
    """|got - want| in the 2-norm over |want|"""
    d = got.detach().double().cpu() - want
    return (d.norm() / want.norm()).item()


# Tolerances in the 2-norm.  Forward: three bf16 roundings (n, h, y) of at most 2^-9 each, n's and
# h's carried through products of random sign: under 3 * 2^-9.  Backward: the same for dy's
# products (dz, dn, dx), and z from E4M3 codes, an error of at most 2^-4 of |z| and 2^-4 / sqrt 3
# in the mean, which an activation of slope about 1 passes on to h and act'(z): under 2^-4.
@pytest.mark.gpu
@pytest.mark.parametrize("rows,width,hidden,act", [(257, 256, 1024, "gelu_tanh"), (1000, 520, 2056, "silu"),
                                                   (64, 128, 96, "relu")])
def test_training_step(rows, width, hidden, act):
    import torch
    from mlp_block import MlpBlock
    b = MlpBlock(width, hidden, act, seed=3)
    r = torch.Generator("cpu").manual_seed(4)
    x = torch.randn(rows, width, generator=r).bfloat16().cuda()
    dy = torch.randn(rows, width, generator=r).bfloat16().cuda()
    y = b.forward(x, keep=True)
    dx = b.backward(dy)
    torch.cuda.synchronize()
    want, x64, p = block64(b, x, act)
    assert rel(y, want.detach()) < 3 * 2.0 ** -9
    want.backward(dy.double().cpu())
    assert rel(b.grads["b2"], p["b2"].grad) < 2.0 ** -16
    for got, w, what in [(dx, x64.grad, "dx")] + [(b.grads[k], p[k].grad, k) for k in ("w2", "b1", "w1", "gamma", "beta")]:
        assert rel(got, w) < 2.0 ** -4, what


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 13])
def test_decoding_step(rows):
    """The rows of a batch and the same rows alone: within the roundings of the forward pass."""
    import torch
    from mlp_block import MlpBlock
    b = MlpBlock(512, 2048, "gelu_tanh", seed=5)
    x = torch.randn(rows, 512, generator=torch.Generator("cpu").manual_seed(6)).bfloat16().cuda()
    y = b.forward(x)
    torch.cuda.synchronize()
    assert b.saved is None
    assert rel(y, block64(b, x, "gelu_tanh")[0].detach()) < 3 * 2.0 ** -9
