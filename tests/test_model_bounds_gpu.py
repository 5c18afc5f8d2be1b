"""GPU: the residual joins and the vocabulary's loss through the bounds-checked
build.  Every access of the row-wise kernels, the loss's statistics, factors and
few-token epilogues is tested against its buffer there (the products' operands,
the rows that the norm's gradient stages and the results that leave by boxes move
by bulk and tensor copies, which their sizes and maps bound).  Sizes on and off
every tile, alignment and layout boundary: nothing falls outside, and the results
are the normal build's."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from tiled_fp32_gemm_gb300 import layers, model

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
            for name in model.SIGNATURES:
                m.setitem(layers._functions, name, getattr(handle, name))
            model._point_native()
            got = call()
            torch.cuda.synchronize()
        model._point_native()
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
@pytest.mark.parametrize("n,d,pad", [(1, 1, 0), (1, 8, 0), (3, 255, 1), (37, 1024, 8),
                                     (5, 3001, 0), (33, 5120, 0), (17, 8192, 0), (3, 8191, 3),
                                     (3, 12288, 0), (2, 16400, 0), (3, 20001, 3)])
def test_joins(checked, dt, n, d, pad):
    x, r, dy = rows(n, d, pad, dt, 1), rows(n, d, pad, dt, 2), rows(n, d, pad, dt, 3)
    w, b = torch.ones(d, device="cuda"), torch.zeros(d, device="cuda")
    f = torch.rand(n, device="cuda")
    kw = dict(dropout=0.3, seed=torch.tensor([9], device="cuda"), sequence=4)
    checked(lambda: mt.layer_norm(x, w, b, residual=r, **kw))
    checked(lambda: mt.layer_norm(x))
    checked(lambda: mt.layer_norm_backward(dy, x, w, f, f, dh=r, **kw))
    checked(lambda: mt.layer_norm_backward(dy, x, None, f, f))
    checked(lambda: (mt.dropout(x, 0.3, kw["seed"], residual=r),))
    checked(lambda: (mt.dropout(x, 0.3, kw["seed"]),))


@pytest.mark.parametrize("T,K,V,pad", [(1, 64, 128, 0), (17, 65, 129, 3), (64, 512, 4096, 0),
                                       (130, 1000, 300, 8), (300, 77, 6001, 1),
                                       (513, 130, 16385, 0)])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_losses(checked, T, K, V, pad, trans, dt):
    a = rows(T, K, pad, dt, 1)
    b = rows(V, K, pad, dt, 2) if trans else rows(K, V, pad, dt, 2)
    g = torch.Generator(device="cuda").manual_seed(5)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    target[T // 2] = -100
    loss, lse = mt.linear_cross_entropy(a, b, target, trans_b=trans)
    kw = dict(trans_b=trans, label_smoothing=0.1, z_loss=1e-3)
    checked(lambda: mt.linear_cross_entropy(a, b, target, **kw))
    checked(lambda: mt.linear_cross_entropy_backward(loss, a, b, target, lse, **kw))
    checked(lambda: mt.linear_cross_entropy_backward(loss, a, b, target, lse, trans_b=trans,
                                                     db_dtype=torch.float32))
