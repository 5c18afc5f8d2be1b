"""The residual joins and the vocabulary's loss together: the example's
training and scoring, its gradients against 64 bits, the torch operator
registrations, and native against Python marshalling."""
import importlib.util
import os

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import tiled_fp32_gemm_gb300 as mt
import tiled_fp32_gemm_gb300.torch_ops  # noqa: F401  (registers torch.ops.mt.*)
from test_layer_norm_gpu import mask_by_columns

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location(
        "language_model", os.path.join(ROOT, "examples", "language_model.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_fakes_give_shapes_without_a_gpu():
    with FakeTensorMode():
        x = torch.empty(5, 8, device="cuda", dtype=torch.bfloat16)
        w = torch.empty(8, device="cuda")
        seed = torch.empty(1, device="cuda", dtype=torch.int64)
        y, h, m, r = torch.ops.mt.layer_norm(x, w, w, x, 1e-5, 0.0, None, 0)
        assert tuple(y.shape) == tuple(h.shape) == (5, 8) and tuple(m.shape) == tuple(r.shape) == (5,)
        assert torch.ops.mt.layer_norm(x, w, w, None, 1e-5, 0.0, None, 0)[1].numel() == 0
        assert torch.ops.mt.layer_norm(x, w, w, None, 1e-5, 0.1, seed, 0)[1].shape == (5, 8)
        assert torch.ops.mt.dropout(x, 0.1, seed, 0, None).shape == (5, 8)
        t = torch.empty(5, device="cuda", dtype=torch.int64)
        loss, lse = torch.ops.mt.linear_cross_entropy(x, torch.empty(20, 8, device="cuda"), t,
                                                      True, -100, 0.0, 0.0)
        assert tuple(loss.shape) == tuple(lse.shape) == (5,) and loss.dtype == torch.float32
        with pytest.raises(Exception):
            torch.ops.mt.layer_norm(x, w[:4], w[:4], None, 1e-5, 0.0, None, 0)
        with pytest.raises(Exception):
            torch.ops.mt.linear_cross_entropy(x, torch.empty(20, 9, device="cuda"), t, True, -100,
                                              0.0, 0.0)


@pytest.mark.gpu
def test_example_trains_and_scores(capsys):
    m = example()
    losses = m.main(["--vocab", "512", "--width", "128", "--hidden", "256", "--tokens", "192",
                     "--steps", "6"])
    assert len(losses) == 6 and all(torch.isfinite(torch.tensor(losses)))
    assert "scoring" in capsys.readouterr().out
    model = m.LanguageModel(500, 64, 96, 1)
    t = torch.arange(9, device="cuda")
    together = model.score(t, t + 3)
    alone = torch.cat([model.score(t[i:i + 1], t[i:i + 1] + 3) for i in range(9)])
    # One hidden state's sums do not depend on the tokens beside it.
    assert (together - alone).abs().max() < 1e-4


def reference(model, tokens, targets, seed, z_loss):
    """The example's loss in 64 bits, from its parameters as bf16 holds them."""
    p = {k: v.detach().bfloat16().double().requires_grad_() if k[-2:] in ("w1", "w2", "ed") else
         v.detach().double().requires_grad_() for k, v in model.params.items()}
    width = p["embed"].shape[1]
    branch, h = p["embed"][tokens], 0.0
    for i in range(model.layers + 1):
        keep = mask_by_columns(len(tokens), width, model.dropout, seed, i)
        h = torch.where(keep, branch / (1 - model.dropout), 0.0) + h
        mean = h.mean(1, keepdim=True)
        r = ((h - mean).square().mean(1, keepdim=True) + 1e-5).rsqrt()
        n = (h - mean) * r * p[f"norm{i}.w"] + p[f"norm{i}.b"]
        if i < model.layers:
            z = n @ p[f"{i}.w1"].t() + p[f"{i}.b1"]
            u = z * 0.5 * torch.erfc(-z / 2 ** 0.5)
            branch = u @ p[f"{i}.w2"].t() + p[f"{i}.b2"]
    z = n @ p["embed"].t()
    lse = torch.logsumexp(z, 1)
    live = targets != -100
    loss = lse - z.gather(1, targets.clamp(min=0)[:, None])[:, 0] + z_loss * lse ** 2
    total = torch.where(live, loss, 0.0).sum() / live.sum()
    return total, dict(zip(p, torch.autograd.grad(total, list(p.values()))))


@pytest.mark.gpu
def test_example_gradients_against_64_bits():
    """bf16 stores round each value by at most 2^-8 of it (2^-9.3 in the mean
    square), and a gradient passes at most 7 of them a layer and 5 at the ends,
    forwards and backwards, 19 for two layers: independent, they come to 19^(1/2) *
    2^-9.3 = 0.7 %, all aligned to 19 * 2^-8 = 7.4 %, which is the bound."""
    m = example()
    model = m.LanguageModel(600, 96, 160, 2, dropout=0.2, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    for k, v in model.params.items():
        if k.startswith("norm") or ".b" in k:
            v.data.add_(0.1 * torch.randn(v.shape, generator=g, device="cuda"))
    tokens, targets = m.batch(600, 300, g)
    seed = torch.tensor([11], dtype=torch.int64, device="cuda")
    loss = model.loss(tokens, targets, seed, z_loss=1e-3)
    grads = torch.autograd.grad(loss, list(model.params.values()))
    want, ref = reference(model, tokens, targets, 11, 1e-3)
    assert abs(loss.item() - want.item()) < 19 * 2 ** -8 * abs(want.item())
    for (name, r), got in zip(ref.items(), grads):
        assert (got.double() - r).norm() <= 19 * 2 ** -8 * r.norm(), name


@pytest.mark.gpu
def test_torch_operators_and_their_gradients():
    g = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, r = draw(40, 72).bfloat16().requires_grad_(), draw(40, 72).bfloat16().requires_grad_()
    w, b = draw(72).requires_grad_(), draw(72).requires_grad_()
    seed = torch.tensor([5], dtype=torch.int64, device="cuda")
    dy, dh = draw(40, 72).bfloat16(), draw(40, 72).bfloat16()
    d = lambda *t: [v.detach() for v in t]  # noqa: E731
    for res, p in ((r, 0.0), (r, 0.3), (None, 0.3), (None, 0.0)):
        y, h, mean, rstd = torch.ops.mt.layer_norm(x, w, b, res, 1e-5, p, seed, 7)
        want = mt.layer_norm(*d(x, w, b), residual=None if res is None else res.detach(),
                             dropout=p, seed=seed, sequence=7)
        assert torch.equal(y, want[0]) and torch.equal(rstd, want[3])
        joined = res is not None or p > 0
        outs, given = ((y, h), (dy, dh)) if joined else ((y,), (dy,))
        leaves = (x, w, b) if res is None else (x, w, b, res)
        got = torch.autograd.grad(outs, leaves, given)
        dx, dres, dw, db = mt.layer_norm_backward(dy, *d(want[1], w, mean, rstd),
                                                  dh=dh if joined else None, dropout=p, seed=seed,
                                                  sequence=7)
        for a, c in zip(got, (dx, dw, db, dres)):
            assert torch.equal(a, c)
    y = torch.ops.mt.dropout(x, 0.4, seed, 2, r)
    got = torch.autograd.grad(y, (x, r), dy)
    assert torch.equal(got[0], mt.dropout(dy, 0.4, seed, 2)) and torch.equal(got[1], dy)
    vocab = draw(300, 72).bfloat16().requires_grad_()
    target = torch.arange(40, device="cuda") * 7
    loss, lse = torch.ops.mt.linear_cross_entropy(x, vocab, target, True, -100, 0.1, 1e-3)
    got = torch.autograd.grad(loss.sum(), (x, vocab))
    ref = mt.linear_cross_entropy_backward(torch.ones(40, device="cuda"), *d(x, vocab), target,
                                           lse, trans_b=True, label_smoothing=0.1, z_loss=1e-3)
    assert all(torch.equal(a, c) for a, c in zip(got, ref))


@pytest.mark.gpu
def test_second_derivatives_and_advanced_seeds_raise():
    x = torch.randn(4, 16, device="cuda").requires_grad_()
    w, b = torch.ones(16, device="cuda").requires_grad_(), torch.zeros(16, device="cuda")
    seed = torch.tensor([5], dtype=torch.int64, device="cuda")
    y = torch.ops.mt.layer_norm(x, w, b, None, 1e-5, 0.2, seed, 0)[0]
    dx, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dx.sum(), x)
    for op in (lambda: torch.ops.mt.dropout(x, 0.2, seed, 0, None),
               lambda: torch.ops.mt.layer_norm(x, w, b, None, 1e-5, 0.2, seed, 0)[0]):
        y = op()
        seed.add_(1)
        with pytest.raises(RuntimeError):
            torch.autograd.grad(y.sum(), x)


def test_native_marshalling_leaves_other_operands_to_python():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    spec = importlib.util.spec_from_file_location("mt_torch_binding", build.binding_path())
    native = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(native)
    x, t = torch.ones(2, 3), torch.zeros(2, dtype=torch.int64)
    assert native.layer_norm(x, None, None, None, 1e-5, 0.0, None, 0) is None
    assert native.layer_norm_backward(x, x, None, x, x, None, 0.0, None, 0, True, True) is None
    assert native.dropout(x, 0.5, t, 0, None) is None
    assert native.dropout(1, 2, 3, 4, 5) is None
    assert native.linear_cross_entropy(x, x, t, True, -100, 0.0, 0.0) is None
    assert native.linear_cross_entropy_backward(x, x, x, t, x, True, -100, 0.0, 0.0, True, True,
                                                None) is None
    with pytest.raises(TypeError):
        native.use_model_library(1)


@pytest.mark.gpu
def test_native_and_python_marshalling_agree(monkeypatch):
    """The same calls with and without the native marshalling: same results,
    same refusals."""
    from tiled_fp32_gemm_gb300 import layers
    g = torch.Generator(device="cuda").manual_seed(8)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, r = draw(9, 80).half()[:, :72], draw(9, 72).half()
    w, f = draw(72), torch.rand(9, device="cuda")
    seed = torch.tensor(77, dtype=torch.int64, device="cuda")
    head, target = draw(40, 72).half(), torch.arange(9, device="cuda")
    kw = dict(dropout=0.25, seed=seed, sequence=2 ** 63 + 5)
    calls = [
        lambda: mt.layer_norm(x, w, w, residual=r, **kw),
        lambda: mt.layer_norm(x, None, w.half(), eps=0.5),
        lambda: mt.layer_norm(x.float()),
        lambda: mt.layer_norm(x, w, **kw),
        lambda: mt.layer_norm_backward(r, x, w, f, f, dh=r, **kw),
        lambda: mt.layer_norm_backward(r, x, None, f, f, need_weight=False),
        lambda: mt.layer_norm_backward(r, x, w.half(), f, f, need_bias=False),
        lambda: (mt.dropout(x, 0.5, seed, residual=r),),
        lambda: (mt.dropout(x, 0.0, seed),),
        lambda: mt.linear_cross_entropy(x, head, target, trans_b=True, label_smoothing=0.1),
        lambda: mt.linear_cross_entropy(x, head.t().contiguous(), target, ignore_index=3),
        lambda: mt.linear_cross_entropy_backward(f, x, head, target, f + 5, trans_b=True,
                                                 z_loss=1e-3, db_dtype=torch.float32),
        lambda: mt.linear_cross_entropy_backward(f, x, head, target, f + 5, trans_b=True,
                                                 need_a=False)]
    refusals = [
        lambda: mt.layer_norm(x, w, w.half()), lambda: mt.layer_norm(x, w[:5]),
        lambda: mt.layer_norm(x, eps=-1.0), lambda: mt.layer_norm(x, dropout=0.1),
        lambda: mt.layer_norm(x, dropout=1.0, seed=seed),
        lambda: mt.layer_norm(x, dropout=0.1, seed=seed.int()),
        lambda: mt.layer_norm(x, dropout=0.1, seed=seed, sequence=2 ** 64),
        lambda: mt.layer_norm_backward(r, x, w, f.half(), f), lambda: mt.dropout(x, 0.1, None),
        lambda: mt.dropout(x, -0.1, seed), lambda: mt.dropout(x, 0.1, seed, residual=r[:3]),
        lambda: mt.linear_cross_entropy(x, head, target),
        lambda: mt.linear_cross_entropy(x, head, target.int(), trans_b=True),
        lambda: mt.linear_cross_entropy(x, head, target, trans_b=True, z_loss=float("inf")),
        lambda: mt.linear_cross_entropy(x, head[:0], target, trans_b=True),
        lambda: mt.linear_cross_entropy_backward(f.half(), x, head, target, f, trans_b=True)]
    mt.layer_norm(x)
    assert layers._native is not None
    fast = [c() for c in calls]

    def answer(c):
        try:
            c()
        except Exception as e:
            return type(e), str(e)

    errors = [answer(c) for c in refusals]
    assert all(errors)
    monkeypatch.setattr(layers, "_native", None)
    for want, c in zip(fast, calls):
        got = c()
        assert len(got) == len(want)
        for a, b in zip(want, got):
            if a is None or b is None:
                assert a is b
            else:
                assert a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()
                # Bit for bit: the lse made up above overflows fp16's D.
                assert torch.equal(a.contiguous().view(torch.uint8),
                                   b.contiguous().view(torch.uint8))
    assert [answer(c) for c in refusals] == errors
