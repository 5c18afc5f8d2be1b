"""An output of the torch operators that nothing reads: its gradient is None, and
no zeros are made for it, added or read; the gradients are those of the calls
without it, bit for bit."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from tiled_fp32_gemm_gb300 import torch_ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()


def draws():
    g = torch.Generator(device="cuda").manual_seed(12)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, r, up = (draw(40, 72).bfloat16() for _ in range(3))
    return x.requires_grad_(), r.requires_grad_(), draw(72).requires_grad_(), \
        draw(72).requires_grad_(), up


class Kept(torch.autograd.Function):
    """The identity, whose gradient goes nowhere."""
    @staticmethod
    def forward(ctx, x):
        return x.clone()

    @staticmethod
    def backward(ctx, g):
        return None


def watch(monkeypatch, name):
    """Has torch_ops' call `name` leave its arguments in the list returned."""
    seen, real = [], getattr(torch_ops, name)

    def call(*args, **kw):
        seen.append((args, kw))
        return real(*args, **kw)
    monkeypatch.setattr(torch_ops, name, call)
    return seen


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_layer_norm(monkeypatch, p):
    x, r, w, b, up = draws()
    seed = torch.tensor([5], device="cuda")
    seen = watch(monkeypatch, "layer_norm_backward")
    y, h, mean, rstd = torch.ops.mt.layer_norm(x, w, b, r, 1e-5, p, seed, 7)
    kw = dict(dropout=p, seed=seed, sequence=7)
    d = [t.detach() for t in (h, w, mean, rstd)]
    got = torch.autograd.grad(y, (x, r, w, b), up, retain_graph=True)
    assert seen[-1][1]["dh"] is None
    dx, dres, dw, db = mt.layer_norm_backward(up, *d, **kw)
    assert all(torch.equal(a, c) for a, c in zip(got, (dx, dres, dw, db)))
    # h alone: y's gradient is zero.
    got = torch.autograd.grad(h, (x, r, w, b), up, retain_graph=True)
    dx, dres, dw, db = mt.layer_norm_backward(torch.zeros_like(up), *d, dh=up, **kw)
    assert all(torch.equal(a, c) for a, c in zip(got, (dx, dres, dw, db)))
    assert not dw.any() and not db.any() and torch.equal(dres, up)
    # Both.
    got = torch.autograd.grad((y, h), (x, r, w, b), (up, up))
    want = mt.layer_norm_backward(up, *d, dh=up, **kw)
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_rms_norm(monkeypatch):
    x, r, w, _, up = draws()
    seen = watch(monkeypatch, "rms_norm_backward")
    y, h, rstd = torch.ops.mt.rms_norm(x, w, r, 1e-5)
    d = [t.detach() for t in (h, w, rstd)]
    for outs, given in ((y,), dict(dy=up)), ((h,), dict(dy=torch.zeros_like(up), dh=up)), \
            ((y, h), dict(dy=up, dh=up)):
        got = torch.autograd.grad(outs, (x, r, w), [up] * len(outs), retain_graph=True)
        assert (seen[-1][1]["dh"] is None) == ("dh" not in given)
        dx, dw = mt.rms_norm_backward(given["dy"], *d, dh=given.get("dh"))
        assert all(torch.equal(a, c) for a, c in zip(got, (dx, dx, dw)))


def test_no_zeros_for_the_pre_activation():
    """The linear layer's backward pass, watched by torch's own allocations: none
    but the gradients'."""
    g = torch.Generator(device="cuda").manual_seed(3)
    a, w = (torch.randn(*s, generator=g, device="cuda").bfloat16().requires_grad_()
            for s in ((512, 64), (4096, 64)))
    y, z = torch.ops.mt.linear(a, w, None, None, "gelu", True)
    up = torch.randn(512, 4096, generator=g, device="cuda").bfloat16()
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    grads = torch.autograd.grad(y, (a, w), up)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before < z.numel() * z.element_size()
    want = mt.linear_backward(up, a.detach(), w.detach(), z=z, activation="gelu", trans_b=True,
                              need_bias=False)
    assert all(torch.equal(x, y) for x, y in zip(grads, want))


def test_gradients_that_go_nowhere():
    x, r, w, b, up = draws()
    seed = torch.tensor([5], device="cuda")
    target = torch.zeros(40, dtype=torch.int64, device="cuda")
    m = torch.randn(96, 72, device="cuda").bfloat16().requires_grad_()
    for out in (torch.ops.mt.layer_norm(x, w, b, r, 1e-5, 0.0, None, 0)[0],
                torch.ops.mt.rms_norm(x, w, r, 1e-5)[0],
                torch.ops.mt.linear(x, m, None, None, "silu", True)[0],
                torch.ops.mt.dropout(x, 0.2, seed, 0, r),
                torch.ops.mt.linear_cross_entropy(x, m, target, True, -100, 0.0, 0.0)[0]):
        loss = Kept.apply(out).float().sum() + x.float().sum()
        got, = torch.autograd.grad(loss, x)
        assert torch.equal(got, torch.ones_like(x))
