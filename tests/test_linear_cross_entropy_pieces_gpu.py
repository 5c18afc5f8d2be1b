"""GPU: the vocabulary loss's gradient where it takes the vocabulary in several
pieces whose shares of dA meet in several planes of sums: the first piece writes
them, the others are added to what is there.  Compared with the definition in 64 bits
under the bounds of test_linear_cross_entropy_gpu.py; the same bits each time, and
whichever gradient is asked for."""
import os
import re

import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from test_linear_cross_entropy_gpu import DTYPES, check_grad, operands

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    yield mt.lib()
    torch.cuda.empty_cache()


def plan_of(T, K, V):
    """(pieces, planes): by the sources' limit of a piece, and as many slices as
    there are pairs of SMs for each tile of dA."""
    source = os.path.join(os.path.dirname(mt.__file__), "csrc", "head_loss.cu")
    with open(source) as f:
        limit = 1 << int(re.search(r"kPieceBytes = int64_t\(1\) << (\d+);", f.read()).group(1))
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    most = max(256, limit // (2 * T) // 256 * 256)
    tiles = -(-T // 256) * -(-K // 256)
    return -(-V // most), sms // 2 // tiles


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("trans", [True, False])
@pytest.mark.parametrize("T,K,V", [(4096, 40, 140000), (8192, 64, 70001), (700, 258, 770001)])
def test_pieces_of_the_vocabulary_in_planes(T, K, V, trans, dtype):
    pieces, planes = plan_of(T, K, V)
    assert pieces > 1 and planes > 1
    a, b, target, dloss = operands(T, K, V, DTYPES[dtype], trans)
    target[::7] = -100
    target[1::7] += (V - 1 - target[1::7]) // 2048 * 2048   # the vocabulary's end
    both = check_grad(a, b, target, dloss, trans, smooth=0.1)
    lse = torch.logsumexp(a.double() @ (b.double().t() if trans else b.double()), 1).float()
    kw = dict(trans_b=trans, label_smoothing=0.1)
    for need in ((True, True), (True, False), (False, True)):
        again = mt.linear_cross_entropy_backward(dloss, a, b, target, lse, need_a=need[0],
                                                 need_b=need[1], **kw)
        for x, y in zip(both, again):
            assert y is None or torch.equal(x, y)
