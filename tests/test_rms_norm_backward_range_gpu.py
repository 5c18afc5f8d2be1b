"""GPU: mt_rms_norm_backward where h is far from 1 and its reciprocal norm as
far on the other side: xhat is of size 1 all the same, and the gradient is
right as long as it fits fp32, whatever kernel the row's width takes.

Tolerances as in the operator's own tests: s |dx| + 8 u |terms| + 80 u of the
mean's spread (u = 2^-24, s half a step of the storage type); dweight 32 u of
the sum of absolute values of its five terms."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


@pytest.mark.parametrize("dt", sorted(STEP, key=str))
@pytest.mark.parametrize("d", [64, 1001, 2048, 8192, 12288, 20000])
@pytest.mark.parametrize("size", [2e-19, 1e-10, 1e10, 5e18])
@pytest.mark.parametrize("gradient", [1e-12, 1.0, 1e3])
@pytest.mark.parametrize("carried", [False, True])
def test_rows_of_any_size(dt, d, size, gradient, carried):
    g = torch.Generator(device="cuda").manual_seed(d)
    draw = lambda s: (torch.randn(5, d, generator=g, device="cuda") * s).to(dt)  # noqa: E731
    h, dy = draw(size), draw(gradient)
    dh = draw(gradient / size) if carried else None
    w = 1 + 0.25 * torch.randn(d, generator=g, device="cuda")
    r = (1 / h.double().square().mean(1).sqrt()).float()
    dx, dw = mt.rms_norm_backward(dy, h, w, r, dh=dh)
    R = r.double()[:, None]
    X, G = h.double() * R, dy.double() * w.double()
    want = R * (G - X * (G * X).mean(1, keepdim=True))
    spread = R * X.abs() * (G * X).abs().mean(1, keepdim=True)
    terms = (R * G).abs() + spread
    if carried:
        want = want + dh.double()
        terms = terms + dh.double().abs()
    err = (dx.double() - want).abs()
    assert (err <= STEP[dt] * want.abs() + 8 * U * terms + 80 * U * spread + 2.0 ** -126).all()
    t = dy.double() * X
    assert ((dw.double() - t.sum(0)).abs() <= 32 * U * t.abs().sum(0)).all()
