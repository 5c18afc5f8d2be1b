"""GPU: rows of zeros through the norm and its gradient, with eps and without:
y and its 8-bit form are zeros, the scale is the smallest one, and without an
eps r is 0, so that the row's gradient is what reaches h directly and the
weight's gradient is the other rows'."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu

DTYPES = [torch.float16, torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("d", [1, 48, 1001, 4096, 17000])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("weighted", [False, True])
def test_zeros_stay_zeros(dt, d, eps, weighted):
    x = torch.ones(3, d, dtype=dt, device="cuda")
    x[1] = 0
    w = torch.full((d,), 2.0, device="cuda") if weighted else None
    size = 2.0 if weighted else 1.0
    y, _, r = mt.rms_norm(x, w, eps=eps)
    assert (y[1] == 0).all()
    assert r[1].item() == (0.0 if eps == 0 else pytest.approx(eps ** -0.5, rel=1e-6))
    q, scale, _, r8 = mt.rms_norm(x, w, eps=eps, out_dtype=torch.float8_e4m3fn)
    assert (q[1].float() == 0).all() and scale[1].item() == mt.MT_SCALE_MIN
    assert torch.equal(r8, r)
    for i in (0, 2):                     # the others as they are: 1 / sqrt(1 + eps) is 1 in 16 bits
        assert ((y[i].double() - size).abs() <= 1e-5).all()
        assert ((q[i].double() - 448) == 0).all()
    # Adding x and its negative gives the same row.
    y2, h, r2 = mt.rms_norm(x, w, residual=torch.where(x == 0, x, -x), eps=0.0)
    assert (h == 0).all() and (y2 == 0).all() and (r2 == 0).all()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("d", [1, 48, 1001, 4096, 17000])
def test_gradient_of_a_row_of_zeros_is_the_carried_one(dt, d):
    g = torch.Generator(device="cuda").manual_seed(d)
    x, dy, dh = (torch.randn(5, d, generator=g, device="cuda").to(dt) for _ in range(3))
    x[2] = 0
    _, _, r = mt.rms_norm(x, None, eps=0.0)
    dx, dw = mt.rms_norm_backward(dy, x, None, r, dh=dh)
    assert torch.equal(dx[2], dh[2])
    keep = [0, 1, 3, 4]
    _, others = mt.rms_norm_backward(dy[keep], x[keep], None, r[keep], dh=dh[keep])
    assert dw.isfinite().all() and dx.isfinite().all()
    # One more term, zero, in a sum of four: at most two roundings each.
    terms = (dy.double() * x.double() * r.double()[:, None]).abs().sum(0)
    assert ((dw - others).abs().double() <= 8 * 2.0 ** -24 * terms).all()
