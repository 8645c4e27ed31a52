"""A gated feed-forward block, trained and then served, on this library.

    h = act(x Wg^T) * (x Wu^T)        gated_matmul
    y = h Wd^T                        matmul (down projection, packed)

Training: a few steps of gradient descent towards a fixed random teacher, with
every product and gradient in the library's kernels (the optimiser's update is
plain torch).  Serving: the trained weights are quantised to 4 bits with group
scales, packed once, and single tokens go through matmul_w4g_gated and
matmul_w4g.

    python examples/feed_forward.py [--tokens 1024] [--width 512] [--hidden 1536] [--steps 30]

Prints the loss per step and the 4-bit block's distance from the 16-bit one.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dense_gemm_preshuffle_gb300 as gp  # noqa: E402


class FeedForward:
    """Wg, Wu [hidden, width] and Wd [width, hidden] in bf16; fp32 master copies for the optimiser."""

    def __init__(self, width: int, hidden: int, seed: int, act: str = "silu"):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        new = lambda r, c: torch.randn((r, c), generator=gen, device="cuda") / c ** 0.5  # noqa: E731
        self.master = [new(hidden, width), new(hidden, width), new(width, hidden)]
        self.width, self.hidden, self.act = width, hidden, act
        self.refresh()

    def refresh(self):
        self.Wg, self.Wu, self.Wd = (w.to(torch.bfloat16) for w in self.master)
        self.Wd_packed = gp.preshuffle_b(self.Wd, "bf16")

    def forward(self, x):
        h = gp.gated_matmul(x, self.Wg, self.Wu, act=self.act)
        return h, gp.matmul(h, self.Wd_packed, "bf16", self.width, self.hidden)

    def step(self, x, target, lr: float) -> float:
        """One step on the mean squared error; returns the loss before it."""
        h, y = self.forward(x)
        e = y.float() - target.float()
        dy = (e * (2.0 / e.numel())).to(torch.bfloat16)
        # y = h Wd^T: dh = dy Wd and dWd = dy^T h, each a product with its right operand packed
        dh = gp.matmul(dy, gp.preshuffle_b(self.Wd.t().contiguous(), "bf16"), "bf16", self.hidden, self.width)
        dWd = gp.matmul(dy.t().contiguous(), gp.preshuffle_b(h.t().contiguous(), "bf16"), "bf16", self.hidden,
                        x.shape[0])
        _, dWg, dWu = gp.gated_matmul_backward(x, self.Wg, self.Wu, dh, act=self.act, need_dA=False)
        for w, g in zip(self.master, (dWg, dWu, dWd)):
            w.sub_(lr * g.float())
        self.refresh()
        return float(e.square().mean())


def quantize(W, group: int):
    """Round a weight matrix to 4 bits: codes (two per byte), scales and zero points per group of `group` values."""
    N, K = W.shape
    g = W.float().reshape(N, K // group, group)
    lo, hi = g.amin(dim=2).clamp(max=0.0), g.amax(dim=2).clamp(min=0.0)
    scale = ((hi - lo) / 15.0).clamp(min=1e-8).to(torch.bfloat16)
    zero = (-lo / scale.float()).round().clamp(0, 15)
    q = (g / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15).to(torch.uint8).reshape(N, K)
    return q[:, 0::2] | (q[:, 1::2] << 4), scale, zero.to(torch.uint8)


class FeedForward4Bit:
    """The block with 4-bit weights, packed once, for a few tokens at a time."""

    def __init__(self, block: FeedForward, group: int = 128):
        self.Wg, self.Wu, self.Wd = (gp.preshuffle_w4g(c.contiguous(), s.contiguous(), group, zeros=z.contiguous())
                                     for c, s, z in (quantize(w, group) for w in (block.Wg, block.Wu, block.Wd)))
        self.act = block.act
        torch.cuda.synchronize()  # the weights are constant from here on

    def __call__(self, x):
        h = gp.matmul_w4g_gated(x, self.Wg, self.Wu, act=self.act, b_constant=True)
        return gp.matmul_w4g(h, self.Wd, b_constant=True)


def run(tokens: int = 1024, width: int = 512, hidden: int = 1536, steps: int = 30, lr: float = 60.0, seed: int = 0):
    """Returns (losses, relative distance of the 4-bit block's outputs from the 16-bit one's)."""
    gen = torch.Generator(device="cuda").manual_seed(seed + 7)
    teacher, block = FeedForward(width, hidden, seed + 1), FeedForward(width, hidden, seed + 2)
    x = torch.randn((tokens, width), generator=gen, device="cuda").to(torch.bfloat16)
    target = teacher.forward(x)[1]
    losses = [block.step(x, target, lr) for _ in range(steps)]
    served = FeedForward4Bit(block)
    token = x[:1]
    y, y4 = block.forward(token)[1].float(), served(token).float()
    return losses, float((y4 - y).norm() / y.norm())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1536)
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    gp.load_library()
    losses, off = run(a.tokens, a.width, a.hidden, a.steps)
    for i, v in enumerate(losses):
        print(f"step {i:3d}  loss {v:.5f}")
    print(f"one token through the 4-bit block: {off:.3f} relative distance from the 16-bit one")
    status = gp.gemm_last_device_status()
    assert status == 0, gp.gemm_status_string(status)


if __name__ == "__main__":
    main()
