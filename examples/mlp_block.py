"""The MLP block of a transformer layer on the library's operators:

    n = layernorm(x) * gamma + beta        z = n W1^T + b1        y = act(z) W2^T + b2 + x

Training keeps, per layer, x, the norm's statistics, n and z as block-scaled E4M3 codes (1.03
bytes per element); h = act(z) is made again from the codes for W2's gradient.  A decoding step
is the same forward pass on one or a few rows, with nothing kept.

    python examples/mlp_block.py [--rows 4096 --width 4096 --hidden 16384 --act gelu_tanh]
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import dense_blas3_gemm_amd as lib  # noqa: E402


class MlpBlock:
    """Weights in bf16 ([out][in]), biases and norm weights and all their gradients in fp32."""

    def __init__(self, width: int, hidden: int, act: str = "gelu_tanh", device: int = 0, seed: int = 0):
        self.g, self.act, self.dev = lib.Gemm(device), act, torch.device("cuda", device)
        r = torch.Generator("cpu").manual_seed(seed)
        rand = lambda *s, std: (torch.randn(*s, generator=r) * std).to(self.dev)  # noqa: E731
        self.gamma, self.beta = 1 + rand(width, std=0.1), rand(width, std=0.1)
        self.w1, self.b1 = rand(hidden, width, std=width ** -0.5).bfloat16(), rand(hidden, std=0.1)
        self.w2, self.b2 = rand(width, hidden, std=hidden ** -0.5).bfloat16(), rand(width, std=0.1)
        self.grads = {k: torch.empty(getattr(self, k).shape, device=self.dev)
                      for k in ("gamma", "beta", "w1", "b1", "w2", "b2")}
        self.saved = None

    def _new(self, *shape, dtype=torch.bfloat16):
        return torch.empty(*shape, device=self.dev, dtype=dtype)

    def forward(self, x, keep: bool = False):
        """y of x [rows][width]; keep: for a backward pass."""
        g, rows, hidden = self.g, x.shape[0], self.w1.shape[0]
        n, h, y = self._new(*x.shape), self._new(rows, hidden), self._new(*x.shape)
        mean = rstd = codes = scales = None
        if keep:
            mean, rstd = self._new(rows, dtype=torch.float32), self._new(rows, dtype=torch.float32)
            codes = self._new(rows, hidden, dtype=torch.uint8)
            scales = self._new(rows, (hidden + 31) // 32, dtype=torch.uint8)
        g.layernorm(x, n, self.gamma, self.beta, mean=mean, rstd=rstd)
        g.run_act(n, self.w1, h, transB=1, bias=self.b1, act=self.act, z=codes, z_scales=scales)
        g.run_act(h, self.w2, y, transB=1, bias=self.b2, residual=x)
        self.saved = (x, n, mean, rstd, codes, scales) if keep else None
        return y

    def backward(self, dy):
        """dx of dy, for the kept forward pass; fills self.grads."""
        g, d = self.g, self.grads
        x, n, mean, rstd, codes, scales = self.saved
        rows, hidden = codes.shape
        h, dz = self._new(rows, hidden), self._new(rows, hidden)
        dn, dx = self._new(*x.shape), self._new(*x.shape)
        g.act_grad_mx(codes, scales, self.act, h=h)
        g(dy, h, d["w2"], transA=1)
        g(torch.ones(1, rows, device=self.dev, dtype=torch.bfloat16), dy, d["b2"].view(1, -1))
        g.run_dact(dy, self.w2, dz, codes, scales, act=self.act, dbias=d["b1"])
        g(dz, n, d["w1"], transA=1)
        g(dz, self.w1, dn)
        g.layernorm_grad(dn, x, mean, rstd, dx, self.gamma, d["gamma"], d["beta"], residual=dy)
        self.saved = None
        return dx


def _seconds(f, steps: int) -> float:
    f()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(steps):
        f()
    torch.cuda.synchronize()
    return (time.perf_counter() - t) / steps


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--rows", type=int, default=4096)
    p.add_argument("--width", type=int, default=4096)
    p.add_argument("--hidden", type=int, default=16384)
    p.add_argument("--act", default="gelu_tanh", choices=lib.ACTS)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    block = MlpBlock(a.width, a.hidden, a.act)
    x = torch.randn(a.rows, a.width, device=block.dev).bfloat16()
    dy = torch.randn(a.rows, a.width, device=block.dev).bfloat16()
    t = _seconds(lambda: (block.forward(x, keep=True), block.backward(dy)), a.steps)
    flops = 12.0 * a.rows * a.width * a.hidden  # six products
    print(f"training step, {a.rows} rows: {t * 1e3:.3f} ms, {flops / t / 1e12:.0f} TFLOP/s")
    for rows in (1, 16):
        one = x[:rows]
        t = _seconds(lambda: block.forward(one), 10 * a.steps)
        moved = 4.0 * a.width * a.hidden  # both weights
        print(f"decoding step, {rows} row(s): {t * 1e6:.1f} us, weights at {moved / t / 1e12:.2f} TB/s")


if __name__ == "__main__":
    main()
