"""GPU: the feed-forward operators through the bounds-checked build.

Every access of the row-wise kernels (norm, its gradient, the gradient of an
activation), the copies of unaligned operands and the products' epilogues is
tested against its buffer there (operands of the products, and the rows the
norm's gradient stages, arrive by bulk and tensor copies that their maps and
sizes bound).  Sizes on and off every tile, alignment and layout boundary:
nothing falls outside, and the results are the normal build's."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from tiled_fp32_gemm_gb300 import layers

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def libraries():
    from tiled_fp32_gemm_gb300 import build
    build.build_many([False, True])
    mt.bounds_status(mt.checked_lib())


@pytest.fixture
def checked(monkeypatch):
    """Runs a call through both builds; the checked one's record must stay
    empty and its results be the same."""
    def run(call):
        want = call()
        handle = mt.checked_lib()
        with monkeypatch.context() as m:
            for name in layers.SIGNATURES:
                m.setitem(layers._functions, name, getattr(handle, name))
            layers._point_native()
            got = call()
            torch.cuda.synchronize()
        layers._point_native()
        status = mt.bounds_status(handle)
        assert status["count"] == 0, status
        for w, g in zip(want, got):
            if w is not None:
                assert torch.equal(w.view(torch.uint8), g.view(torch.uint8))
    return run


def rows(n, d, pad, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, d + pad, generator=g, device="cuda").to(dt)[:, :d]


@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
@pytest.mark.parametrize("n,d,pad", [(1, 8, 0), (3, 255, 1), (37, 1024, 8), (5, 3001, 0),
                                     (33, 5120, 0), (17, 8192, 0), (3, 12288, 0),
                                     (2, 16400, 0), (3, 20001, 3)])
def test_norms(checked, dt, n, d, pad):
    x, r, dy = rows(n, d, pad, dt, 1), rows(n, d, pad, dt, 2), rows(n, d, pad, dt, 3)
    w = torch.ones(d, device="cuda")
    checked(lambda: mt.rms_norm(x, w, residual=r))
    checked(lambda: mt.rms_norm(x, w, out_dtype=torch.float8_e4m3fn))
    rstd = torch.rand(n, device="cuda")
    checked(lambda: mt.rms_norm_backward(dy, x, w, rstd, dh=r))
    checked(lambda: mt.rms_norm_backward(dy, x, None, rstd))


@pytest.mark.parametrize("M,N,K,pad", [(1, 128, 64, 0), (17, 129, 65, 3), (64, 4096, 512, 0),
                                       (130, 300, 1000, 8), (500, 1001, 77, 1),
                                       (2305, 2561, 130, 0)])
@pytest.mark.parametrize("trans", [False, True])
def test_products_and_gradients(checked, M, N, K, pad, trans):
    dt = torch.bfloat16
    a, dy, z = rows(M, K, pad, dt, 1), rows(M, N, pad, dt, 2), rows(M, N, 2 * pad, dt, 3)
    b = rows(N, K, pad, dt, 4) if trans else rows(K, N, pad, dt, 4)
    bias = torch.ones(N, device="cuda")
    checked(lambda: mt.linear(a, b, bias=bias, activation="gelu", residual=z, trans_b=trans,
                              preact=True))
    checked(lambda: mt.linear_backward(dy, a, b, z=z, activation="silu", trans_b=trans,
                                       db_dtype=torch.float32))
    checked(lambda: mt.linear_backward(dy, a, b, trans_b=trans))
    if trans:
        q, p = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
        s, t = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
        checked(lambda: (mt.linear(q, p, bias=bias, trans_b=True, scale_a=s, scale_b=t,
                                   out_dtype=torch.float32),))
