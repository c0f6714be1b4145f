"""Layer norm's gradient at the widest row that the entry points take, 2^31 - 1 columns (one workgroup
walks it twice: some ten seconds)."""
import pytest

pytestmark = pytest.mark.gpu
N = 2 ** 31 - 1


def spread(t, cuts):
    """Largest distance of t from value v between columns a and b, over the (a, b, v) of `cuts`."""
    worst = 0.0
    for a, b, v in cuts:
        for i in range(a, b, 1 << 28):
            worst = max(worst, (t[0, i:min(b, i + (1 << 28))].float() - v).abs().max().item())
    return worst

def test_widest_row(gpu):
    import torch
    half, three = N // 2, N // 2 + N // 4
    x = torch.ones(1, N, dtype=torch.bfloat16, device="cuda")
    x[0, half:] = -1
    dy = torch.zeros_like(x)
    dy[0, half:three] = 1
    dx = torch.full_like(x, float("nan"))
    mean, rstd = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    gpu.layernorm_grad(dy, x, mean, rstd, dx)
    torch.cuda.synchronize()
    # dx = dy - 1/4 + x/4, all but 2^-30 of it
    assert spread(dx, [(0, half, 0.0), (half, three, 0.5), (three, N, -0.5)]) < 2.0 ** -9
