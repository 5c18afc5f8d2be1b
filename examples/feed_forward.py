"""A transformer's feed-forward block on the library, trained and served.

    h = x + residual;  n = rms_norm(h);  u = gelu(n W1 + b1);  y = u W2 + b2 + h

``train`` takes a few steps of gradient descent on one block (bf16 weights
with fp32 copies, the gradients through ``rms_norm_backward`` and
``linear_backward``), ``serve`` runs the trained block on 8-bit rows: the norm
writes e4m3 with a scale per row, which the first product reads against an
e4m3 weight with a scale per column; the second product adds the residual.

    python examples/feed_forward.py [--width 1024] [--hidden 4096] [--tokens 512] [--steps 20]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_fp32_gemm_gb300 as mt  # noqa: E402

EPS = 1e-5


class FeedForward:
    """The block's parameters: fp32 copies that the optimiser steps, and the
    bf16 weights that the products read.  Weights are stored N x K."""

    def __init__(self, width, hidden, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.master = {"norm": torch.ones(width, device="cuda"),
                       "w1": draw(hidden, width) / math.sqrt(width),
                       "b1": torch.zeros(hidden, device="cuda"),
                       "w2": draw(width, hidden) / math.sqrt(hidden),
                       "b2": torch.zeros(width, device="cuda")}
        self.refresh()

    def refresh(self):
        self.w1 = self.master["w1"].bfloat16()
        self.w2 = self.master["w2"].bfloat16()

    def forward(self, x, residual):
        """(y, what the backward pass needs)."""
        p = self.master
        n, h, rstd = mt.rms_norm(x, p["norm"], residual=residual, eps=EPS)
        u, z = mt.linear(n, self.w1, bias=p["b1"], activation="gelu", trans_b=True, preact=True)
        y = mt.linear(u, self.w2, bias=p["b2"], residual=h, trans_b=True)
        return y, (n, h, rstd, u, z)

    def backward(self, dy, saved):
        """(gradient of x and of the residual, gradients of the parameters)."""
        n, h, rstd, u, z = saved
        du, dw2, db2 = mt.linear_backward(dy, u, self.w2, trans_b=True, db_dtype=torch.float32)
        dn, dw1, db1 = mt.linear_backward(du, n, self.w1, z=z, activation="gelu", trans_b=True,
                                          db_dtype=torch.float32)
        dx, dnorm = mt.rms_norm_backward(dn, h, self.master["norm"], rstd, dh=dy)
        return dx, {"norm": dnorm, "w1": dw1, "b1": db1, "w2": dw2, "b2": db2}

    def step(self, grads, rate):
        for name, g in grads.items():
            self.master[name].sub_(g, alpha=rate)
        self.refresh()


def quantise(w):
    """(e4m3 rows, float32 scale per row) of a weight, laid out once."""
    scale = (w.abs().amax(dim=1) / mt.MT_E4M3_MAX).clamp(min=mt.MT_SCALE_MIN)
    return (w / scale[:, None]).to(torch.float8_e4m3fn), scale


def train(block, x, residual, target, steps, rate):
    """Mean squared error against `target` after each step."""
    losses = []
    for _ in range(steps):
        y, saved = block.forward(x, residual)
        error = y.float() - target
        losses.append(error.square().mean().item())
        dy = (error * (2.0 / error.numel())).bfloat16()
        _, grads = block.backward(dy, saved)
        block.step(grads, rate)
    return losses


class Served:
    """The block for inference: e4m3 first product, bf16 second."""

    def __init__(self, block):
        self.norm, self.b1 = block.master["norm"], block.master["b1"]
        self.w2, self.b2 = block.w2, block.master["b2"]
        self.w1, self.s1 = quantise(block.master["w1"])

    def __call__(self, x, residual):
        q, scale, h, _ = mt.rms_norm(x, self.norm, residual=residual, eps=EPS,
                                     out_dtype=torch.float8_e4m3fn)
        u = mt.linear(q, self.w1, bias=self.b1, activation="gelu", trans_b=True, scale_a=scale,
                      scale_b=self.s1, out_dtype=torch.bfloat16)
        return mt.linear(u, self.w2, bias=self.b2, residual=h, trans_b=True, out=h)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    g = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda n: torch.randn(n, a.width, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, residual = draw(a.tokens), draw(a.tokens)
    teacher = FeedForward(a.width, a.hidden, seed=7)
    target = teacher.forward(x, residual)[0].float()
    block = FeedForward(a.width, a.hidden, seed=3)
    losses = train(block, x, residual, target, a.steps, rate=4.0)
    print(f"training: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")
    served = Served(block)
    for tokens in (1, 16, a.tokens):
        want = block.forward(x[:tokens], residual[:tokens])[0].float()
        got = served(x[:tokens], residual[:tokens]).float()
        rel = ((got - want).norm() / want.norm()).item()
        print(f"serving {tokens} token(s) in 8 bits: {rel:.4f} of the 16-bit output's norm off")
    if mt.mt_check_device_status(0) != mt.MT_OK:
        raise SystemExit("device status reported a failure")
    return losses


if __name__ == "__main__":
    main()
