"""GPU: the feed-forward operators on matrices past 2^31 elements (offsets
that do not fit 32 bits): the first and last rows against the definition in
64 bits.  Tolerances as in the operators' own tests."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu

U, S = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 60 GB")
    yield mt.lib()
    torch.cuda.empty_cache()


def ends(rows):
    return torch.cat([torch.arange(3), torch.arange(rows - 3, rows)]).cuda()


@pytest.mark.parametrize("rows,d", [(265000, 8192), (265001, 8191), (110000, 20000)])
def test_norm_and_its_gradient(rows, d):
    assert rows * d > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, d, generator=g, device="cuda", dtype=torch.bfloat16)
    y, _, rstd = mt.rms_norm(x, None, eps=1e-5)
    at = ends(rows)
    X = x[at].double()
    r = torch.rsqrt(X.square().mean(1) + 1e-5)
    assert ((rstd[at].double() - r).abs() <= 64 * U * r).all()
    want = X * r[:, None]
    assert ((y[at].double() - want).abs() <= (S + 70 * U) * want.abs()).all()
    dx, _ = mt.rms_norm_backward(y, x, None, rstd, need_weight=False)
    D, H = y[at].double(), X * rstd[at].double()[:, None]
    R = rstd[at].double()[:, None]
    spread = R * H.abs() * (D * H).abs().mean(1, keepdim=True)
    want = R * (D - H * (D * H).mean(1, keepdim=True))
    tol = S * want.abs() + 88 * U * spread + 8 * U * (R * D).abs()
    assert ((dx[at].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("N", [2048, 2047])
def test_linear_and_its_gradient(N):
    M, K = 1060000, 32
    assert M * N > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    a = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    b = torch.randn(N, K, generator=g, device="cuda", dtype=torch.bfloat16)
    y = mt.linear(a, b, activation="relu", trans_b=True)
    at = ends(M)
    A, B = a[at].double(), b.double()
    W = A.abs() @ B.abs().t()
    want = (A @ B.t()).clamp(min=0)
    assert ((y[at].double() - want).abs() <= 6e-5 * W + S * want).all()
    da, db, dbias = mt.linear_backward(y, a, b, z=y, activation="relu", trans_b=True,
                                       need_b=False)
    Z = y[at].double()
    want = Z @ B                       # relu's gradient of y at y is y
    W = Z @ B.abs()
    assert ((da[at].double() - want).abs() <= (S + 6e-5) * W + S * want.abs()).all()
    total = torch.zeros(N, dtype=torch.float64, device="cuda")
    for rows in y.split(100000):
        total += rows.double().sum(0)
    # 1.06 M terms, all of one sign: at most M / 128 deep in one thread's sum.
    assert ((dbias.double() - total).abs() <= M / 128 * U * total).all()
    assert mt.mt_check_device_status(0) == mt.MT_OK
