"""GPU: tokens without a target whose logits overflow the exponential (their D is a
row of zeros all the same, not the NaN of infinity times zero), or are NaN."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from test_linear_cross_entropy_gpu import DTYPES, check_grad, check_loss, logits, operands

pytestmark = pytest.mark.gpu

# Few tokens (the split kernel) and a batch (pairs).
BATCHES = [3, 300]


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


def ignored(T, dtype):
    a, b, target, dloss = operands(T, 64, 6000, DTYPES[dtype], True)
    target[1] = -100
    return a.clone(), b, target, dloss


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T", BATCHES)
def test_logits_past_the_exponential(T, dtype):
    a, b, target, dloss = ignored(T, dtype)
    a[1] *= 200
    top = logits(a, b, True)[0][1].amax()
    assert top > 128 and top.float().exp().isinf()
    check_loss(a, b, target, True)
    da, db = check_grad(a, b, target, dloss, True)
    assert da.isfinite().all() and db.isfinite().all()
    # Nor does it matter what the row's lse and gradient hold.
    _, lse = mt.linear_cross_entropy(a, b, target, trans_b=True)
    want = mt.linear_cross_entropy_backward(dloss, a, b, target, lse, trans_b=True)
    lse[1], dloss[1] = float("nan"), float("inf")
    got = mt.linear_cross_entropy_backward(dloss, a, b, target, lse, trans_b=True)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("T", BATCHES)
def test_logits_of_nan(T, dtype):
    """The row's dA is zeros and the others' keep their bits (its row of A enters
    dB's sums times zero, so dB is not asked for)."""
    a, b, target, dloss = ignored(T, dtype)
    _, lse = mt.linear_cross_entropy(a, b, target, trans_b=True)
    want, _ = mt.linear_cross_entropy_backward(dloss, a, b, target, lse, trans_b=True,
                                               need_b=False)
    a[1, 5] = float("nan")
    a[1, 9] = float("inf")
    loss, lse = mt.linear_cross_entropy(a, b, target, trans_b=True)
    assert loss[1] == 0 and lse[1].isnan() and loss.isfinite().all()
    got, _ = mt.linear_cross_entropy_backward(dloss, a, b, target, lse, trans_b=True,
                                              need_b=False)
    assert not got[1].any() and torch.equal(got, want)
