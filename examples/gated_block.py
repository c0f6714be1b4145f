"""A gated feed-forward block on the library's operators:

    G = x Wg^T    U = x Wu^T    H = act(G) U    y = H Wd^T + x

Training keeps x, G and U, and makes H again in the backward pass, in the product that runs back
through it; Wg and Wu lie side by side in one buffer, so that dx and their gradient are one product
each.  A serving step runs the same block in bf16, or with its weights as 8-bit integers with a
factor for each output channel and its activations quantised row by row on the way.

    python examples/gated_block.py [--rows 4096 --width 4096 --hidden 10944 --act silu]
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import dense_blas3_gemm_amd as lib  # noqa: E402


class GatedBlock:
    """Weights in bf16 ([out][in], the gate's and the other projection's in `w`), gradients in fp32."""

    def __init__(self, width: int, hidden: int, act: str = "silu", device: int = 0, seed: int = 0):
        self.g, self.act, self.dev, self.hidden = lib.Gemm(device), act, torch.device("cuda", device), hidden
        r = torch.Generator("cpu").manual_seed(seed)
        rand = lambda *s: (torch.randn(*s, generator=r) * s[1] ** -0.5).to(self.dev).bfloat16()  # noqa: E731
        self.w, self.wd = rand(2 * hidden, width), rand(width, hidden)
        self.grads = {k: torch.empty(getattr(self, k).shape, device=self.dev) for k in ("w", "wd")}
        self.saved = None
        self.q = None

    def _new(self, *shape, dtype=torch.bfloat16):
        return torch.empty(*shape, device=self.dev, dtype=dtype)

    def forward(self, x, keep: bool = False):
        """y of x [rows][width]; keep: for a backward pass."""
        rows, n = x.shape[0], self.hidden
        h, y = self._new(rows, n), self._new(*x.shape)
        gate, up = (self._new(rows, n), self._new(rows, n)) if keep else (None, None)
        self.g.run_gated(x, self.w[:n], self.w[n:], h, transB=1, act=self.act, g=gate, u=up)
        self.g.run_act(h, self.wd, y, transB=1, residual=x)
        self.saved = (x, gate, up) if keep else None
        return y

    def backward(self, dy):
        """dx of dy, for the kept forward pass; fills self.grads."""
        x, gate, up = self.saved
        rows, n = gate.shape
        d, h, dx = self._new(rows, 2 * n), self._new(rows, n), self._new(*x.shape)
        self.g.run_dgated(dy, self.wd, gate, up, d[:, :n], d[:, n:], act=self.act, h=h)
        self.g(dy, h, self.grads["wd"], transA=1)
        self.g(d, x, self.grads["w"], transA=1)
        dx.copy_(dy)
        self.g(d, self.w, dx, beta=1.0)
        self.saved = None
        return dx

    def quantize(self):
        """The weights as 8-bit integers, once."""
        def one(w):
            q, s = self._new(*w.shape, dtype=torch.int8), self._new(w.shape[0], dtype=torch.float32)
            self.g.quantize_i8(w, q, s)
            return q, s
        self.q = one(self.w) + one(self.wd)

    def forward_i8(self, x):
        """y on the quantised weights."""
        w, sw, wd, sd = self.q
        rows, n = x.shape[0], self.hidden
        xq, xs = self._new(*x.shape, dtype=torch.int8), self._new(rows, dtype=torch.float32)
        hq, hs = self._new(rows, n, dtype=torch.int8), self._new(rows, dtype=torch.float32)
        h, y = self._new(rows, n), self._new(*x.shape)
        self.g.quantize_i8(x, xq, xs)
        self.g.run_gated_i8(xq, xs, w[:n], sw[:n], w[n:], sw[n:], h, transB=1, act=self.act)
        self.g.quantize_i8(h, hq, hs)
        self.g.run_i8(hq, hs, wd, sd, y, transB=1, residual=x)
        return y


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
    p.add_argument("--hidden", type=int, default=10944)
    p.add_argument("--act", default="silu", choices=lib.ACTS)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    block = GatedBlock(a.width, a.hidden, a.act)
    x = torch.randn(a.rows, a.width, device=block.dev).bfloat16()
    dy = torch.randn(a.rows, a.width, device=block.dev).bfloat16()
    t = _seconds(lambda: (block.forward(x, keep=True), block.backward(dy)), a.steps)
    flops = 18.0 * a.rows * a.width * a.hidden  # nine products
    print(f"training step, {a.rows} rows: {t * 1e3:.3f} ms, {flops / t / 1e12:.0f} TFLOP/s")
    block.quantize()
    weights = 3.0 * a.width * a.hidden
    for rows in (1, 16, a.rows):
        one = x[:rows]
        for name, f, size in (("bf16", block.forward, 2), ("int8", block.forward_i8, 1)):
            t = _seconds(lambda: f(one), (10 if rows < 64 else 1) * a.steps)
            print(f"serving step, {rows} row(s), {name}: {t * 1e6:.1f} us, weights at {size * weights / t / 1e12:.2f} TB/s, "
                  f"{2 * rows * weights / t / 1e12:.0f} T operations/s")


if __name__ == "__main__":
    main()
