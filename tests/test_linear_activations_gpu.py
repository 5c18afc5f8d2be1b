"""GPU: mt_linear's activations by themselves, against 64 bits.

With K == 0 the pre-activation is the bias exactly, so nothing of a product's
rounding hides the activation's own: each result has to be right to its own
digits, in the tails too, where gelu and silu fall towards zero.

Tolerances (u = 2^-24), of the result:
* fp32: gelu's fit is within 1.7 u, its argument and evaluation within 6 u,
  expf within 2 ulp (4 u), and four more roundings: 16 u.  silu's expf, sum,
  reciprocal (1 ulp) and products: 11 u.  The tanh form's logistic takes exp of
  v = 2 u(z), good to 4.5 u of itself: 5 |v| u more.  What is below the type's
  normal range has an absolute grid: 2^-126.
* 16-bit: 2^-15, and the result's own rounding.  The exponentials flush to
  zero what is below 2^-110; fp16 rounds on a grid of 2^-24 at the bottom.
"""
import numpy as np
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
FLOOR = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -110, torch.float32: 2.0 ** -126}


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


def points():
    """Both tails of each activation, the middle, and the types' ends: 8192
    values."""
    z = np.concatenate([np.linspace(-14, 14, 4000), np.linspace(-105, 105, 3000),
                        np.geomspace(1e-30, 1, 590), -np.geomspace(1e-30, 1, 590),
                        [0.0, -0.0, 1e4, -1e4, 6e4, -6e4, 1e15, -1e15, 1e30, -1e30,
                         3e38, -3e38]])
    assert z.size == 8192
    return torch.from_numpy(z.astype(np.float32)).cuda()


def tanh_argument(z):
    return 2 * (2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)


def definition(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / 2 ** 0.5)
    if act == "gelu_tanh":                       # (1 + tanh u) / 2 is the logistic of 2 u
        return z * torch.sigmoid(tanh_argument(z))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("inputs", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("f32", [False, True])
def test_activation_keeps_its_digits(act, inputs, f32):
    z = points()
    a = torch.empty(2, 0, dtype=inputs, device="cuda")
    b = torch.empty(0, z.numel(), dtype=inputs, device="cuda")
    dt = torch.float32 if f32 else inputs
    y = mt.linear(a, b, bias=z, activation=act, out_dtype=dt)
    assert y.dtype == dt and torch.equal(y[0], y[1])
    Z = z.double()
    want = definition(Z, act)
    if f32:
        rel = torch.full_like(want, 16 * U)
        if act == "gelu_tanh":
            rel += 5 * tanh_argument(Z).abs() * U
    else:
        rel = torch.full_like(want, 2.0 ** -15) + HALF_STEP[dt] * (1 + 2.0 ** -15)
    # What a result past the type's largest value becomes, infinity, is the
    # rounding's; the points past it are fp16's alone.
    fits = want.abs() < torch.finfo(dt).max * (1 - 2.0 ** -9)
    err = (y[0].double() - want).abs()
    bad = fits & ~(err <= rel * want.abs() + FLOOR[dt])
    worst = (err / want.abs().clamp(min=FLOOR[dt]))[bad]
    assert not bad.any(), (z[bad][:8], worst[:8])
    assert (y[0][~fits].abs() >= torch.finfo(dt).max * (1 - 2.0 ** -8)).all()
