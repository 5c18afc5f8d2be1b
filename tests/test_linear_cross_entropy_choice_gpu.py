"""GPU: the vocabulary's loss and its gradient on both sides of the sizes at which
its logits go from the split kernel to CTA pairs (1280 values of K, a seventh as
many tiles as SMs, 128 tokens)."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from test_linear_cross_entropy_gpu import check_grad, check_loss, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


@pytest.mark.parametrize("trans", [True, False])
@pytest.mark.parametrize("T,K,V", [(129, 1280, 700), (129, 1281, 700), (128, 1280, 700),
                                   (257, 1999, 1001), (520, 1281, 1793), (513, 1500, 1792),
                                   (600, 2056, 2500)])
def test_either_side(T, K, V, trans):
    dt = torch.float16 if K % 2 else torch.bfloat16
    a, b, target, dloss = operands(T, K, V, dt, trans)
    target[::5] = -100
    check_loss(a, b, target, trans, 0.1, 1e-3)
    check_grad(a, b, target, dloss, trans, 0.1, 1e-3)
