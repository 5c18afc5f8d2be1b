"""The feed-forward operators together: the example's training and serving
paths, and the torch operator registrations with their gradients."""
import importlib.util
import os

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import tiled_fp32_gemm_gb300 as mt
import tiled_fp32_gemm_gb300.torch_ops  # noqa: F401  (registers torch.ops.mt.*)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_fakes_give_shapes_without_a_gpu():
    with FakeTensorMode():
        a = torch.empty(5, 8, device="cuda", dtype=torch.bfloat16)
        w = torch.empty(12, 8, device="cuda", dtype=torch.bfloat16)
        y, z = torch.ops.mt.linear(a, w, None, None, "gelu", True)
        assert tuple(y.shape) == tuple(z.shape) == (5, 12) and y.dtype == torch.bfloat16
        y, z = torch.ops.mt.linear(a, w.t().contiguous(), None, None, "none", False)
        assert tuple(y.shape) == (5, 12) and tuple(z.shape) == (0,)
        with pytest.raises(Exception):
            torch.ops.mt.linear(a, w, None, None, "gelu", False)
        n, h, r = torch.ops.mt.rms_norm(a, torch.empty(8, device="cuda"), a, 1e-5)
        assert tuple(n.shape) == tuple(h.shape) == (5, 8) and tuple(r.shape) == (5,)
        with pytest.raises(Exception):
            torch.ops.mt.rms_norm(a, torch.empty(9, device="cuda"), None, 1e-5)


@pytest.mark.gpu
def test_example_trains_and_serves(capsys):
    losses = example().main(["--width", "256", "--hidden", "640", "--tokens", "96", "--steps",
                             "15"])
    assert losses[-1] < 0.5 * losses[0]
    # 8-bit rows and weights: each rounded to 2^-4 of a value at most, 2^-5.3
    # in the mean square; the residual, which is not rounded, is the larger
    # part of the output.
    for line in capsys.readouterr().out.splitlines():
        if line.startswith("serving"):
            assert float(line.split(": ")[1].split()[0]) < 2 ** -4


@pytest.mark.gpu
def test_block_gradient_against_differences():
    """The example's backward pass against central differences of the block
    in 64 bits, along random directions of every parameter and input."""
    m = example()
    block = m.FeedForward(48, 80, seed=2)
    g = torch.Generator(device="cuda").manual_seed(5)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, res, dy = draw(24, 48).bfloat16(), draw(24, 48).bfloat16(), draw(24, 48).bfloat16()
    y, saved = block.forward(x, res)
    dx, grads = block.backward(dy, saved)
    p = {k: v.double() for k, v in block.master.items()}
    p["w1"], p["w2"] = block.w1.double(), block.w2.double()

    def f(q, x, res):
        h = x + res
        n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + m.EPS) * q["norm"]
        z = n @ q["w1"].t() + q["b1"]
        u = z * 0.5 * torch.erfc(-z / 2 ** 0.5)
        return ((u @ q["w2"].t() + q["b2"] + h) * dy.double()).sum()

    for _ in range(4):
        d = {k: draw(*v.shape).double() for k, v in p.items()}
        ex, er = draw(24, 48).double(), draw(24, 48).double()
        t = 1e-5
        at = lambda s: f({k: v + s * d[k] for k, v in p.items()}, x.double() + s * ex,  # noqa: E731
                         res.double() + s * er)
        num = (at(t) - at(-t)) / (2 * t)
        terms = [(dx.double() * (ex + er)).flatten()]
        terms += [(grads[k].double() * d[k]).flatten() for k in grads]
        terms = torch.cat(terms)
        # bf16 intermediates (n, h, u, z, du, dz, dn, dx), each a relative
        # error of 2^-9, independent from element to element: ten standard
        # deviations of the terms' random sum, over eight roundings.
        assert abs(terms.sum() - num) <= 10 * 2 ** -9 * 8 ** 0.5 * terms.square().sum().sqrt()


@pytest.mark.gpu
def test_operators_match_the_binding_and_differentiate():
    g = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    a, w = draw(40, 64).bfloat16().requires_grad_(), draw(96, 64).bfloat16().requires_grad_()
    bias, res = draw(96).requires_grad_(), draw(40, 96).bfloat16().requires_grad_()
    for act in ("none", "silu"):
        y, _ = torch.ops.mt.linear(a, w, bias, res, act, True)
        want = mt.linear(a.detach(), w.detach(), bias=bias.detach(), residual=res.detach(),
                         activation=act, trans_b=True, preact=True)
        assert torch.equal(y.detach(), want[0])
        dy = draw(40, 96).bfloat16()
        got = torch.autograd.grad(y, (a, w, bias, res), dy)
        ref = mt.linear_backward(dy, a.detach(), w.detach(), z=want[1], activation=act,
                                 trans_b=True)
        for i in range(3):
            assert torch.equal(got[i], ref[i])
        assert torch.equal(got[3], dy)
    x, nw = draw(40, 64).bfloat16().requires_grad_(), draw(64).requires_grad_()
    r2 = draw(40, 64).bfloat16().requires_grad_()
    y, h, rstd = torch.ops.mt.rms_norm(x, nw, r2, 1e-5)
    dy, dh = draw(40, 64).bfloat16(), draw(40, 64).bfloat16()
    got = torch.autograd.grad((y, h), (x, nw, r2), (dy, dh))
    ref = mt.rms_norm_backward(dy, h.detach(), nw.detach(), rstd.detach(), dh=dh)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[2], ref[0])
    assert torch.equal(got[1], ref[1])
    y, h, rstd = torch.ops.mt.rms_norm(x, nw, None, 1e-5)
    got = torch.autograd.grad(y, (x, nw), dy)
    ref = mt.rms_norm_backward(dy, x.detach(), nw.detach(), rstd.detach())
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_native_marshalling_is_built_and_leaves_other_operands_to_python():
    """build() makes it for the installed torch; what it does not take (here:
    host tensors, numbers) it answers with None, never with an error."""
    from tiled_fp32_gemm_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("mt_torch_binding", build.binding_path())
    native = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(native)
    x = torch.ones(2, 3)
    assert native.rms_norm(x, None, None, 1e-5, None) is None
    assert native.rms_norm(1, 2, 3, 4, 5) is None
    assert native.rms_norm_backward(x, x, None, x, None, True) is None
    assert native.linear(x, x, None, 0, None, True, None, None, None, False) is None
    assert native.linear_backward(x, x, x, None, 0, True, True, True, True, None) is None
    with pytest.raises(TypeError):
        native.use_library(1)


@pytest.mark.gpu
def test_native_and_python_marshalling_agree(monkeypatch):
    """The same calls with and without the native marshalling: same results,
    same refusals."""
    from tiled_fp32_gemm_gb300 import layers
    g = torch.Generator(device="cuda").manual_seed(8)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, r = draw(9, 80).half()[:, :72], draw(9, 72).half()
    w, n = draw(40, 72).half(), draw(72)
    q, s = w.to(torch.float8_e4m3fn), torch.rand(40, device="cuda")
    z, dy, bias = draw(9, 40).half(), draw(9, 48).half()[:, :40], draw(40)
    rstd = torch.rand(9, device="cuda")
    calls = [
        lambda: mt.rms_norm(x, n, residual=r),
        lambda: mt.rms_norm(x, None, eps=0.5),
        lambda: mt.rms_norm(x, n.half(), out_dtype=torch.float8_e4m3fn),
        lambda: mt.rms_norm_backward(r, x, n, rstd, dh=r),
        lambda: mt.rms_norm_backward(r, x, None, rstd, need_weight=False),
        lambda: mt.linear(x, w, bias=bias, activation="gelu", residual=z, trans_b=True,
                          preact=True),
        lambda: (mt.linear(x, w.t().contiguous(), out_dtype=torch.float32),),
        lambda: (mt.linear(q, q, trans_b=True, scale_a=s, scale_b=s),),
        lambda: mt.linear_backward(dy, x, w, z=z, activation="silu", trans_b=True),
        lambda: mt.linear_backward(dy, x, w.t().contiguous(), need_a=False,
                                   db_dtype=torch.float32),
    ]
    refusals = [lambda: mt.rms_norm(x, n, eps=-1.0), lambda: mt.rms_norm(x, n[:5]),
                lambda: mt.rms_norm(x, n, out_dtype=torch.bfloat16),
                lambda: mt.linear(x, w), lambda: mt.linear(x, w.bfloat16(), trans_b=True),
                lambda: mt.linear(x, w, trans_b=True, residual=z[:3]),
                lambda: mt.linear_backward(dy, x, w, activation="relu", trans_b=True),
                lambda: mt.rms_norm_backward(r, x, n, rstd.half())]
    mt.rms_norm(x, n)
    assert layers._native is not None
    fast = [f() for f in calls]

    def answer(f):
        try:
            f()
        except Exception as e:
            return type(e), str(e)

    errors = [answer(f) for f in refusals]
    assert all(errors)
    monkeypatch.setattr(layers, "_native", None)
    for want, f in zip(fast, calls):
        got = f()
        assert len(got) == len(want)
        for a, b in zip(want, got):
            if a is None or b is None:
                assert a is b
            else:
                assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()
                assert torch.equal(a.float(), b.float())
    assert [answer(f) for f in refusals] == errors
