"""GPU: mt_linear_backward against its formula in 64 bits, and the formula
against differences of the layer's definition.

Tolerance: dz is rounded once to the storage type (s: half a step, plus 16 u
for the derivative's fp32 evaluation, whose values are below 1.13 and whose
terms are below 2), and each product's fp32 sums are within 5e-5 of the sum
of absolute values, so a gradient is within (s + 5e-5 + 32 u) * W plus its
own rounding, W the product of absolute values.  dbias adds unrounded terms:
(32 + 300) u of the sum of |dY| * 2.
"""
import numpy as np
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: U}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


def stored(g, rows, cols, pitch, dt, scale=1.0):
    buf = torch.full((rows, pitch), float("nan"))
    buf[:, :cols] = torch.randn(rows, cols, generator=g) * scale
    return buf.to(dt).cuda()[:, :cols]


def slope(z, act):
    """Derivative of each activation in 64 bits."""
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return 0.5 * torch.erfc(-z / 2 ** 0.5) + z * torch.exp(-z * z / 2) / (2 * np.pi) ** 0.5
    if act == "gelu_tanh":
        c = (2 / np.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def check(dy, a, b, z, act, trans, **kw):
    da, db, dbias = mt.linear_backward(dy, a, b, z=z, activation=act, trans_b=trans, **kw)
    assert mt.mt_check_device_status(0) == mt.MT_OK
    D = dy.double()
    dz = D * slope(z.double(), act) if z is not None else D
    A, B = a.double(), b.double()
    B = B.t() if trans else B
    s = STEP[dy.dtype]
    lost = s if act != "none" else 0.0
    # Entries of dz below fp16's normal range round on its fixed grid.
    grid = 2.0 ** -25 if dy.dtype == torch.float16 else 2.0 ** -130

    def near(got, want, W, ones, dt):
        so = STEP[dt]
        tol = (lost + 5e-5 + 32 * U) * W + grid * ones
        tiny = 2.0 ** -25 if dt == torch.float16 else 2.0 ** -130
        err = (got.double() - want).abs()
        assert got.dtype == dt and got.shape == want.shape
        assert (err <= tol * (1 + so) + so * want.abs() + tiny).all(), (err - tol).max()

    size = D.abs() * 1.13
    near(da, dz @ B.t(), size @ B.t().abs(), torch.ones_like(D) @ B.t().abs(), dy.dtype)
    want, W, ones = A.t() @ dz, A.t().abs() @ size, A.t().abs() @ torch.ones_like(D)
    if trans:
        want, W, ones = want.t(), W.t(), ones.t()
    near(db, want, W, ones, kw.get("db_dtype") or dy.dtype)
    err = (dbias.double() - dz.sum(0)).abs()
    assert dbias.dtype == torch.float32 and (err <= 664 * U * D.abs().sum(0)).all()
    return da, db, dbias


@pytest.mark.parametrize("dt", sorted(DTYPES))
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 128, 64), (1, 1, 1), (3, 1000, 70), (17, 130, 129),
                                   (64, 512, 1024), (100, 72, 80), (129, 257, 513),
                                   (512, 640, 256), (1000, 264, 300), (2500, 65, 64)])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("act", ACTS)
def test_matches_the_formula(dt, trans, M, N, K, pad, act):
    g = torch.Generator().manual_seed(M + 7 * N + 13 * K + pad)
    t = DTYPES[dt]
    dy = stored(g, M, N, N + pad, t)
    z = stored(g, M, N, N + 2 * pad, t, 2.0) if act != "none" else None
    a = stored(g, M, K, K + pad, t)
    shape = (N, K) if trans else (K, N)
    b = stored(g, *shape, shape[1] + pad, t, K ** -0.5)
    check(dy, a, b, z, act, trans, db_dtype=torch.float32 if M % 2 else None)


@pytest.mark.parametrize("dt", sorted(DTYPES))
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("M,N,K", [(2400, 2305, 2561), (2305, 2305, 2305)])
def test_tiles_that_fill_the_gpu(dt, trans, act, M, N, K):
    g = torch.Generator().manual_seed(M + trans)
    t = DTYPES[dt]
    dy, a = stored(g, M, N, N + 7, t), stored(g, M, K, K + 7, t)
    z = stored(g, M, N, N, t, 2.0) if act != "none" else None
    shape = (N, K) if trans else (K, N)
    check(dy, a, stored(g, *shape, shape[1], t, K ** -0.5), z, act, trans,
          db_dtype=torch.float32 if M % 2 else None)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", sorted(DTYPES))
def test_derivatives_over_their_range(act, dt):
    """Pre-activations from -300 to 300 and the type's largest values: every
    derivative finite and right."""
    t = DTYPES[dt]
    z = torch.cat([torch.linspace(-300, 300, 3000), torch.tensor([6e4, -6e4, 0.0, -0.0])])
    z = z.to(t).cuda()[None, :].repeat(2, 1)
    if act == "none":
        z = None
    dy = torch.ones(2, 3004, dtype=t, device="cuda")
    eye = torch.eye(2, dtype=t, device="cuda")
    b = torch.zeros(2, 3004, dtype=t, device="cuda")
    da, db, dbias = mt.linear_backward(dy, eye, b, z=z, activation=act)
    want = slope(z.double(), act)[0] if z is not None else torch.ones(3004).cuda()
    assert ((dbias.double() / 2 - want).abs() <= 32 * U * (1 + want.abs())).all()
    assert ((db[0].double() - want).abs() <=
            STEP[t] * want.abs() + 32 * U + 2.0 ** -25).all()
    assert (da == 0).all()


@pytest.mark.parametrize("act", ACTS)
def test_formula_against_differences(act):
    """Central differences of sum(act(A B + bias) * dY) in 64 bits along a
    random direction, against the gradients of the kernels."""
    g = torch.Generator().manual_seed(11)
    M, N, K = 40, 72, 56
    a, b = stored(g, M, K, K, torch.float16), stored(g, K, N, N, torch.float16, K ** -0.5)
    dy = stored(g, M, N, N, torch.float16)
    bias = torch.randn(N, generator=g).cuda()
    y, z = mt.linear(a, b, bias=bias, activation=act, preact=True, out_dtype=torch.float16)
    da, db, dbias = mt.linear_backward(dy, a, b, z=z, activation=act, db_dtype=torch.float32)

    def act64(v):
        if act == "relu":
            return v.clamp(min=0)
        if act == "gelu":
            return v * 0.5 * torch.erfc(-v / 2 ** 0.5)
        if act == "gelu_tanh":
            return 0.5 * v * (1 + torch.tanh((2 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3)))
        return v * torch.sigmoid(v) if act == "silu" else v

    A, B, c, D = a.double(), b.double(), bias.double(), dy.double()
    for _ in range(3):
        u, v, w = (torch.randn(*s, generator=g, dtype=torch.float64).cuda()
                   for s in ((M, K), (K, N), (N,)))

        def f(t):
            return (act64((A + t * u) @ (B + t * v) + c + t * w) * D).sum()

        t = 1e-5
        num = (f(t) - f(-t)) / (2 * t)
        got = (da.double() * u).sum() + (db.double() * v).sum() + (dbias.double() * w).sum()
        # The gradients' roundings (da, dz and z to fp16) are independent
        # from element to element: 8 of their standard deviations, plus, for
        # relu's kink, the few pre-activations a step of t or z's rounding
        # carries across zero.
        step = 2.0 ** -11
        size = ((da.double() * u).square().sum() + (db.double() * v).square().sum()
                + (dbias.double() * w).square().sum()
                + (D.square() * (u @ B + A @ v + w).square()).sum()).sqrt()
        assert abs(got - num) <= 8 * step * size + 1e-6 * size


@pytest.mark.parametrize("M", [0, 7])
def test_empty_sums_are_zeros(M):
    a = torch.ones(M, 24, dtype=torch.float16, device="cuda")
    b = torch.ones(24, 40, dtype=torch.float16, device="cuda")
    dy = torch.ones(M, 40, dtype=torch.float16, device="cuda")
    da, db, dbias = mt.linear_backward(dy, a, b)
    assert da.shape == (M, 24) and (db == M).all() and (dbias == M).all()
    da, db, dbias = mt.linear_backward(dy[:, :0], a, b[:, :0])
    assert (da == 0).all() and db.shape == (24, 0) and dbias.shape == (0,)
    da, db, dbias = mt.linear_backward(dy, a[:, :0], b[:0])
    assert da.shape == (M, 0) and db.shape == (0, 40) and (dbias == M).all()


def test_parts_on_their_own_and_the_same_bits():
    g = torch.Generator().manual_seed(2)
    a, b = stored(g, 300, 520, 520, torch.bfloat16), stored(g, 700, 520, 520, torch.bfloat16)
    dy, z = stored(g, 300, 700, 703, torch.bfloat16), stored(g, 300, 700, 700, torch.bfloat16)
    want = mt.linear_backward(dy, a, b, z=z, activation="gelu", trans_b=True)
    for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)):
        got = mt.linear_backward(dy, a, b, z=z, activation="gelu", trans_b=True, need_a=need[0],
                                 need_b=need[1], need_bias=need[2])
        for w, x, n in zip(want, got, need):
            assert torch.equal(w, x) if n else x is None


def test_nan_reaches_its_row_and_column():
    a = torch.ones(30, 40, dtype=torch.bfloat16, device="cuda")
    b = torch.ones(40, 50, dtype=torch.bfloat16, device="cuda")
    dy = torch.ones(30, 50, dtype=torch.bfloat16, device="cuda")
    z = torch.ones_like(dy)
    z[4, 9] = float("nan")
    for act in ACTS[1:]:
        da, db, dbias = mt.linear_backward(dy, a, b, z=z, activation=act)
        assert da[4].isnan().all() and db[:, 9].isnan().all() and dbias[9].isnan()
        assert da.isnan().sum() == 40 and db.isnan().sum() == 40 and dbias.isnan().sum() == 1


def test_refusals():
    a = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        mt.linear_backward(dy, a, b, activation="gelu")           # no pre-activation
    with pytest.raises(TypeError):
        mt.linear_backward(dy.half(), a, b)
    with pytest.raises(TypeError):
        mt.linear_backward(dy, a, b, db_dtype=torch.float16)
    with pytest.raises(ValueError):
        mt.linear_backward(dy, a, b, trans_b=True)
    with pytest.raises(ValueError):
        mt.linear_backward(dy[:3], a, b)
    with pytest.raises(ValueError):
        mt.linear_backward(dy, a, b, z=dy, activation="swish")
