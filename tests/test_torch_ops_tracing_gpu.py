"""The torch operators traced together, and recomputed by torch's checkpointing: what
eager calls give."""
import pytest
import torch
from torch.utils.checkpoint import checkpoint

import tiled_fp32_gemm_gb300.torch_ops  # noqa: F401  (registers torch.ops.mt.*)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()


def leaves():
    g = torch.Generator(device="cuda").manual_seed(0)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return [t.requires_grad_() for t in (draw(64, 128).bfloat16(), draw(64, 128).bfloat16(),
                                         draw(128), draw(128), draw(256, 128).bfloat16())]


def step(x, r, w, b, m):
    """Every operator once, some outputs read and some not."""
    seed, target = torch.full((1,), 3, device="cuda"), torch.arange(64, device="cuda")
    y, h, _, _ = torch.ops.mt.layer_norm(x, w, b, r, 1e-5, 0.1, seed, 0)
    u, _ = torch.ops.mt.linear(y, m, None, None, "gelu", True)
    n, h2, _ = torch.ops.mt.rms_norm(h, w, torch.ops.mt.dropout(y, 0.2, seed, 1, None), 1e-5)
    n, _, _, _ = torch.ops.mt.layer_norm(n, w, None, h2, 1e-5, 0.0, None, 0)
    loss, _ = torch.ops.mt.linear_cross_entropy(n, m, target, True, -100, 0.0, 1e-3)
    return loss.sum() + u.float().sum()


def test_traced_forwards():
    args = leaves()
    with torch.no_grad():
        want = step(*args)
        assert torch.equal(torch.compile(step, backend="aot_eager")(*args), want)


def test_recomputed_by_a_checkpoint():
    args = leaves()
    want = torch.autograd.grad(step(*args), args)
    got = torch.autograd.grad(checkpoint(step, *args, use_reentrant=False), args)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert want[3].any()


def test_captured_forwards_and_backwards():
    """Warmed up on the side stream, whose graph of autograd is gone by the capture."""
    args = leaves()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in torch.autograd.grad(step(*args), args)]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(step(*args), args)
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
