"""The torch operator of the layer norm without a weight or without a bias: taken as
by the function it registers, with the same gradients."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import tiled_fp32_gemm_gb300 as mt
import tiled_fp32_gemm_gb300.torch_ops  # noqa: F401  (registers torch.ops.mt.*)

FORMS = [(True, False), (False, True), (False, False)]


def test_shapes_without_a_gpu():
    with FakeTensorMode():
        x = torch.empty(5, 8, device="cuda", dtype=torch.bfloat16)
        w = torch.empty(8, device="cuda")
        for weight, bias in FORMS:
            y, h, m, r = torch.ops.mt.layer_norm(x, w if weight else None, w if bias else None, x,
                                                 1e-5, 0.0, None, 0)
            assert tuple(y.shape) == tuple(h.shape) == (5, 8)
            assert tuple(m.shape) == tuple(r.shape) == (5,)
        for weight, bias in ((w[:4], None), (None, w[:4]), (None, x), (w, w[:4])):
            with pytest.raises(Exception):
                torch.ops.mt.layer_norm(x, weight, bias, None, 1e-5, 0.0, None, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("vectors", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("weight,bias", FORMS)
def test_results_and_gradients(weight, bias, p, vectors):
    g = torch.Generator(device="cuda").manual_seed(21)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, r, dy, dh = (draw(33, 72).bfloat16() for _ in range(4))
    w, b = (draw(72).to(vectors).requires_grad_() if there else None for there in (weight, bias))
    x, r = x.requires_grad_(), r.requires_grad_()
    seed = torch.tensor([9], device="cuda")
    y, h, mean, rstd = torch.ops.mt.layer_norm(x, w, b, r, 1e-5, p, seed, 2)
    plain = [None if t is None else t.detach() for t in (x, w, b, r)]
    want = mt.layer_norm(*plain, dropout=p, seed=seed, sequence=2)
    assert all(torch.equal(a, c) for a, c in zip((y, h, mean, rstd), want))
    leaves = [t for t in (x, r, w, b) if t is not None]
    got = torch.autograd.grad((y, h), leaves, (dy, dh))
    dx, dres, dw, db = mt.layer_norm_backward(dy, want[1], plain[1], want[2], want[3], dh=dh,
                                              dropout=p, seed=seed, sequence=2)
    ref = [dx, dres] + [v.to(vectors) for v, t in ((dw, w), (db, b)) if t is not None]
    assert len(got) == len(ref) and all(torch.equal(a, c) for a, c in zip(got, ref))
