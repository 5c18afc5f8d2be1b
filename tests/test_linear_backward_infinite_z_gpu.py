"""GPU: the gradient of `linear` at pre-activations that fp16 (or bf16) could
not hold and stored as infinity: each derivative has its limit there, 0 or 1,
as beside it at the type's largest values."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("pad", [0, 3])
def test_derivatives_at_infinity(act, dt, pad):
    top = torch.finfo(dt).max
    row = torch.tensor([float("inf"), top, -top, float("-inf")] * 10)
    z = torch.zeros(3, 40 + pad)
    z[:, :40] = row
    z = z.to(dt).cuda()[:, :40]
    dy = torch.full((3, 40 + pad), 0.5).to(dt).cuda()[:, :40]
    a = torch.eye(3, 8).to(dt).cuda()
    b = torch.ones(8, 40).to(dt).cuda()
    da, db, dbias = mt.linear_backward(dy, a, b, z=z, activation=act)
    slope = (row > 0).double().cuda()
    assert torch.equal(dbias.double(), 1.5 * slope)
    assert torch.equal(db[:3].double(), 0.5 * slope.expand(3, 40))
    assert (da.double() == 0.5 * slope.sum()).all()


def test_a_product_that_passes_fp16_trains_on():
    """z = 2^17 in fp32 is stored as infinity: the gradient is the limit's
    all the same."""
    a = torch.full((4, 64), 32.0, device="cuda").half()
    b = torch.full((64, 8), 64.0, device="cuda").half()
    _, z = mt.linear(a, b, activation="gelu", preact=True)
    assert z.isinf().all()
    da, db, dbias = mt.linear_backward(torch.ones_like(z), a, b, z=z, activation="gelu",
                                       db_dtype=torch.float32)
    assert (dbias == 4).all() and (da == 512).all() and (db == 128).all()
