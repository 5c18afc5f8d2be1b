"""A small residual language model on the library, trained and scored.

    h_0 = drop(E[token]);  h_i = drop(branch_i) + h_(i-1)
    branch_(i+1) = gelu(norm(h_i) W1 + b1) W2 + b2
    loss = cross entropy of norm(h_n) E^T

Each join, its dropout and the layer norm after it are one pass
(``torch.ops.mt.layer_norm``); the logits of the tied embedding's product exist
nowhere (``torch.ops.mt.linear_cross_entropy``).  ``train`` takes a few steps,
captured once in a CUDA graph: the seed in device memory advances with every
replay, so each drops other elements.  ``score`` gives single tokens' log
probabilities.  The task is to predict the token that a fixed permutation sends
each token to.

    python examples/language_model.py [--vocab 4096] [--width 512] [--hidden 2048]
        [--layers 2] [--tokens 1024] [--steps 40] [--dropout 0.1]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_fp32_gemm_gb300 as mt  # noqa: E402
import tiled_fp32_gemm_gb300.torch_ops  # noqa: E402,F401  (registers torch.ops.mt.*)

EPS = 1e-5
IGNORED = -100


class LanguageModel:
    """fp32 parameters, cast to bf16 where a product reads them.  Weights are
    stored N x K; the embedding, V x width, is the head's weight too."""

    def __init__(self, vocab, width, hidden, layers, dropout=0.1, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.dropout, self.layers = dropout, layers
        p = {"embed": draw(vocab, width) / math.sqrt(width)}
        for i in range(layers + 1):
            p[f"norm{i}.w"] = torch.ones(width, device="cuda")
            p[f"norm{i}.b"] = torch.zeros(width, device="cuda")
        for i in range(layers):
            p[f"{i}.w1"] = draw(hidden, width) / math.sqrt(width)
            p[f"{i}.b1"] = torch.zeros(hidden, device="cuda")
            p[f"{i}.w2"] = draw(width, hidden) / math.sqrt(hidden)
            p[f"{i}.b2"] = torch.zeros(width, device="cuda")
        self.params = {k: v.requires_grad_() for k, v in p.items()}

    def hidden(self, tokens, seed=None):
        """(normalised hidden states, the head's weight); seed None: no dropout."""
        p = self.params
        drop = self.dropout if seed is not None else 0.0
        embed = p["embed"].bfloat16()
        branch, stream = embed[tokens], None
        for i in range(self.layers + 1):
            n, h, _, _ = torch.ops.mt.layer_norm(branch, p[f"norm{i}.w"], p[f"norm{i}.b"], stream,
                                                 EPS, drop, seed, i)
            stream = h if h.numel() else branch  # nothing dropped or added: h is the branch
            if i < self.layers:
                u, _ = torch.ops.mt.linear(n, p[f"{i}.w1"].bfloat16(), p[f"{i}.b1"], None, "gelu",
                                           True)
                branch, _ = torch.ops.mt.linear(u, p[f"{i}.w2"].bfloat16(), p[f"{i}.b2"], None,
                                                "none", True)
        return n, embed

    def loss(self, tokens, targets, seed=None, z_loss=1e-4):
        """Mean loss over the tokens that have a target."""
        n, embed = self.hidden(tokens, seed)
        loss, _ = torch.ops.mt.linear_cross_entropy(n, embed, targets, True, IGNORED, 0.0, z_loss)
        return loss.sum() / (targets != IGNORED).sum().clamp(min=1)

    @torch.no_grad()
    def score(self, tokens, targets):
        """Log probability of each target after its token."""
        n, embed = self.hidden(tokens)
        return -mt.linear_cross_entropy(n, embed, targets, trans_b=True)[0]


def batch(vocab, tokens, g):
    """Random tokens and where the permutation sends them, some without a target."""
    t = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    target = (t * 5 + 1) % vocab if vocab % 5 else (t + 1) % vocab
    target[torch.rand(tokens, generator=g, device="cuda") < 0.05] = IGNORED
    return t, target


def train(model, vocab, tokens, steps, rate=0.5):
    """Steps of gradient descent, the losses before each: one warm-up step, then
    replays of one captured step."""
    g = torch.Generator(device="cuda").manual_seed(1)
    token, target = batch(vocab, tokens, g)
    seed = torch.full((1,), 17, dtype=torch.int64, device="cuda")
    params = list(model.params.values())

    def step():
        loss = model.loss(token, target, seed)
        for p, d in zip(params, torch.autograd.grad(loss, params)):
            p.data.add_(d, alpha=-rate)
        seed.add_(1)
        return loss.detach()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        losses = [step().item()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(steps - 1):
        for static, fresh in zip((token, target), batch(vocab, tokens, g)):
            static.copy_(fresh)
        graph.replay()
        losses.append(out.item())
    return losses


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--vocab", type=int, default=4096)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--dropout", type=float, default=0.1)
    a = ap.parse_args(argv)
    model = LanguageModel(a.vocab, a.width, a.hidden, a.layers, a.dropout)
    losses = train(model, a.vocab, a.tokens, a.steps)
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {a.steps} steps")
    g = torch.Generator(device="cuda").manual_seed(2)
    token, target = batch(a.vocab, 64, g)
    each = [model.score(token[i:i + 1], target[i:i + 1]).item() for i in range(4)]
    print("scoring: log probabilities " + ", ".join(f"{v:.3f}" for v in each))
    return losses


if __name__ == "__main__":
    main()
