"""The gated operators together, as examples/gated_block.py uses them, against the same block in
float64 autograd on the values the operators are given."""
import os
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

from test_gpu_mlp_block import ACTS, rel  # noqa: E402

pytestmark = pytest.mark.gpu


def block64(b, x, act):
    """y, and the tensors to differentiate, in float64 on the CPU"""
    w, wd, x = (t.detach().double().cpu().requires_grad_(True) for t in (b.w, b.wd, x))
    n = b.hidden
    return (ACTS[act](x @ w[:n].T) * (x @ w[n:].T)) @ wd.T + x, x, w, wd


# Tolerances in the 2-norm, bf16 half steps of at most 2^-8 of a value (2^-8 / sqrt 3 in the mean).
# Forward: h, carried through a product of random sign, and y.  Backward: G and U as kept, which h, the
# gate and its slope take over (a slope's own slope is under 1), and the roundings of dG, dU, H and
# dx: under five of them on any way.
@pytest.mark.parametrize("rows,width,hidden,act", [(257, 256, 688, "gelu_tanh"), (1000, 520, 1384, "silu"),
                                                   (64, 128, 96, "relu"), (5, 512, 1368, "silu")])
def test_training_step(rows, width, hidden, act):
    import torch
    from gated_block import GatedBlock
    b = GatedBlock(width, hidden, act, seed=3)
    r = torch.Generator("cpu").manual_seed(4)
    x = torch.randn(rows, width, generator=r).bfloat16().cuda()
    dy = torch.randn(rows, width, generator=r).bfloat16().cuda()
    y = b.forward(x, keep=True)
    dx = b.backward(dy)
    torch.cuda.synchronize()
    want, x64, w, wd = block64(b, x, act)
    assert rel(y, want.detach()) < 2 * 2.0 ** -8
    want.backward(dy.double().cpu())
    for got, g, what in ((dx, x64.grad, "dx"), (b.grads["w"], w.grad, "w"), (b.grads["wd"], wd.grad, "wd")):
        assert rel(got, g) < 5 * 2.0 ** -8, what


# 8-bit integers: a row's values are off by up to half of max / 127, at random: of normal values with a
# largest of about 3.5 deviations 3.5 / 254 / sqrt 3 * 2 = 0.016 of the row's norm at most.  The weights
# of either projection and x make two such errors in G and in U, their product four; h (whose largest
# is some ten deviations: 0.05) and Wd two more.  Against the residual's norm that is added to y.
@pytest.mark.parametrize("rows", [1, 13, 300])
def test_serving_steps(rows):
    import torch
    from gated_block import GatedBlock
    b = GatedBlock(512, 1368, "silu", seed=5)
    x = torch.randn(rows, 512, generator=torch.Generator("cpu").manual_seed(6)).bfloat16().cuda()
    y = b.forward(x)
    b.quantize()
    y8 = b.forward_i8(x)
    torch.cuda.synchronize()
    assert b.saved is None
    want = block64(b, x, "silu")[0].detach()
    assert rel(y, want) < 2 * 2.0 ** -8
    assert rel(y8, want) < 4 * 0.016 + 0.05 + 0.016 + 2.0 ** -8
