"""The registered operators' gradients have no gradient of their own: a second
derivative raises, where it would otherwise lose the parts through the kernels
and keep those beside them."""
import pytest
import torch

import tiled_fp32_gemm_gb300.torch_ops  # noqa: F401  (registers torch.ops.mt.*)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()


def leaf(*shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    return torch.randn(*shape, generator=g, device="cuda").to(dtype).requires_grad_()


def linear():
    a, w, res = leaf(16, 64), leaf(96, 64), leaf(16, 96)
    y, _ = torch.ops.mt.linear(a, w, None, res, "silu", True)
    return y, (a, w, res)


def rms_norm():
    x, w, res = leaf(16, 64), leaf(64, dtype=torch.float32), leaf(16, 64)
    y, h, _ = torch.ops.mt.rms_norm(x, w, res, 1e-5)
    return y * h, (x, w, res)


@pytest.mark.parametrize("of", [linear, rms_norm])
def test_second_derivatives_raise(of):
    y, leaves = of()
    first = torch.autograd.grad(y.float().square().sum(), leaves, create_graph=True)
    # A gradient penalty: the first gradients' size, and the loss beside it.
    penalty = sum(g.float().square().sum() for g in first) + leaves[0].float().sum()
    with pytest.raises(RuntimeError, match="once_differentiable"):
        penalty.backward()


@pytest.mark.parametrize("of", [linear, rms_norm])
def test_first_derivatives_are_the_same_with_a_graph(of):
    y, leaves = of()
    dy = torch.ones_like(y)
    plain = torch.autograd.grad(y, leaves, dy, retain_graph=True)
    graph = torch.autograd.grad(y, leaves, dy, create_graph=True)
    for p, g in zip(plain, graph):
        assert torch.equal(p, g.detach())
