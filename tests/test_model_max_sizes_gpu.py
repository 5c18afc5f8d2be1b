"""GPU: the residual joins and the vocabulary's loss on operands past 2^31
elements: rows or columns at the far end get what a call on them alone gives, or
their definition in 64 bits."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    torch.cuda.empty_cache()
    yield mt.lib()
    torch.cuda.empty_cache()


def far(rows, d, seed):
    """rows x d bf16 values, made a block of rows at a time."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    for part in x.split(1 << 16):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return x


@pytest.mark.parametrize("rows,d", [(270000, 8192), (131100, 16392), (270100, 8191)])
def test_norms_and_dropout(rows, d):
    x, r = far(rows, d, 1), far(rows, d, 2)
    w, b = torch.rand(d, device="cuda"), torch.rand(d, device="cuda")
    y, h, mean, rstd = mt.layer_norm(x, w, b, residual=r)
    tail = slice(rows - 5, rows)
    for got, want in zip((y, h, mean, rstd), mt.layer_norm(x[tail].clone(), w, b,
                                                           residual=r[tail].clone())):
        assert torch.equal(got[tail], want)
    dx, _, dw, db = mt.layer_norm_backward(x, h, w, mean, rstd, dh=r)
    want = mt.layer_norm_backward(x[tail].clone(), h[tail].clone(), w, mean[tail].clone(),
                                  rstd[tail].clone(), dh=r[tail].clone())
    assert torch.equal(dx[tail], want[0])
    # Sums over all rows, at most rows / 8 + 64 deep.
    total = sum(p.double().sum(0) for p in x.split(1 << 14))
    size = sum(p.double().abs().sum(0) for p in x.split(1 << 14))
    assert ((db.double() - total).abs() <= (rows / 8 + 64) * 2.0 ** -24 * size).all()
    del dx, y, h
    seed = torch.tensor([3], dtype=torch.int64, device="cuda")
    y = mt.dropout(x, 0.5, seed, residual=r)
    keep = mt.dropout(torch.ones_like(x), 0.5, seed)[tail] != 0
    want = (torch.where(keep, 2.0 * x[tail].float(), 0.0) + r[tail].float()).bfloat16()
    assert torch.equal(y[tail], want)


@pytest.mark.parametrize("trans", [True, False])
def test_loss_of_a_large_weight(trans):
    """Weight and its gradient past 2^31 elements, targets at its far end."""
    T, K, V = 5, 8192, 270000
    a = far(T, K, 1) / 64
    b = far(V, K, 2) if trans else far(K, V, 2)
    target = torch.tensor([V - 1, V - 300, 0, 1, V // 2], device="cuda")
    loss, lse = mt.linear_cross_entropy(a, b, target, trans_b=trans)
    A = a.double()
    z = torch.cat([A @ p.double().t() for p in b.split(1 << 14)], 1) if trans else \
        torch.cat([A @ p.double() for p in b.split(1 << 14, dim=1)], 1)
    want = torch.logsumexp(z, 1)
    # Sums of products within 5e-5 of their absolute values, which are 64 here.
    assert (lse - want).abs().max() < 5e-5 * 80
    assert (loss - want + z.gather(1, target[:, None])[:, 0]).abs().max() < 1e-4 * 80
    da, db = mt.linear_cross_entropy_backward(torch.ones(T, device="cuda"), a, b, target, lse,
                                              trans_b=trans)
    D = (z - lse.double()[:, None]).exp().scatter_add(1, target[:, None], -A.new_ones(T, 1))
    for cols in (slice(V - 400, V), slice(0, 300), slice(V // 2 - 3, V // 2 + 3)):
        got = db[cols] if trans else db[:, cols].t()
        ref = D[:, cols].t() @ A
        size = D[:, cols].t().abs() @ A.abs()
        # p within 5e-5 * 80, D and the result rounded to 2^-8 each.
        assert ((got.double() - ref).abs() <= (2 ** -7 + 5e-3) * size + 1e-12).all()


def test_loss_of_many_tokens():
    """More tokens than a piece of D holds at once for a wide vocabulary, and
    D past 2^31 elements in all."""
    T, K, V = 600000, 64, 4096
    a, b = far(T, K, 3), far(V, K, 4) / 8
    g = torch.Generator(device="cuda").manual_seed(5)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    loss, lse = mt.linear_cross_entropy(a, b, target, trans_b=True)
    dloss = torch.full((T,), 1e-3, device="cuda")
    da, db = mt.linear_cross_entropy_backward(dloss, a, b, target, lse, trans_b=True)
    at = torch.cat([torch.arange(300), torch.arange(T // 2, T // 2 + 40),
                    torch.arange(T - 300, T)]).cuda()
    alone, alse = mt.linear_cross_entropy(a[at], b, target[at], trans_b=True)
    assert (alone - loss[at]).abs().max() < 1e-4 and (alse - lse[at]).abs().max() < 1e-4
    z = a[at].double() @ b.double().t()
    D = 1e-3 * ((z - lse[at].double()[:, None]).exp()
                .scatter_add(1, target[at][:, None], -z.new_ones(len(at), 1)))
    ref, size = D @ b.double(), D.abs() @ b.double().abs()
    assert ((da[at].double() - ref).abs() <= (2 ** -7 + 5e-3) * size + 1e-12).all()
    total = torch.zeros(V, K, dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(total)
    for i in range(0, T, 50000):
        s = slice(i, i + 50000)
        D = 1e-3 * ((a[s].double() @ b.double().t() - lse[s].double()[:, None]).exp()
                    .scatter_add(1, target[s][:, None], -total.new_ones(len(lse[s]), 1)))
        total += D.t() @ a[s].double()
        bound += D.t().abs() @ a[s].double().abs()
    assert ((db.double() - total).abs() <= (2 ** -7 + 5e-3) * bound).all()
