"""GPU: the scale that the vocabulary loss's gradient holds D in takes dloss's own
digits out of the rounding to 16 bits: a loss averaged over its tokens, whatever
their number, gives the gradients of a power of two for dloss, times a factor.

Tolerances (u = 2^-24, norms of dB in fp32).  The scaled D of two dloss differ by 4 u,
which moves an entry across a rounding border with a probability of at most 8 u over a
step of 2^-8 (bf16), and then by 2^-8 of it: (8 u 2^8)^(1/2) 2^-8 = 2^-14.5 of D in
norm; the products' sums truncate alike, but for what moved, and their factor is
rounded once: 2^-13 for all.  A factor rounded with D is off by up to 2^-8 (bf16) or
2^-11 (fp16), by 3.4e-3 and 4.3e-4 for the one below."""
import pytest
import torch

import test_linear_cross_entropy_gpu as loss_tests
import tiled_fp32_gemm_gb300 as mt
from test_linear_cross_entropy_gpu import DTYPES, check_grad, operands

pytestmark = pytest.mark.gpu

FACTOR = 1.0037e-3   # 1.0278 * 2^-10
BIG = 1 << 36        # (T + 256) * K * V from which bf16 is scaled too


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    yield mt.lib()
    torch.cuda.empty_cache()


def db_of(value, a, b, target, lse, **kw):
    dloss = torch.full((len(target),), value, device="cuda")
    return mt.linear_cross_entropy_backward(dloss, a, b, target, lse, db_dtype=torch.float32,
                                            **kw)


# fp16 at every size; bf16 where the scale's kernels do not show.  Slices of dA,
# both products on pairs, operands that are copied, one token.
CASES = [("f16", 1, 64, 500, True), ("f16", 300, 72, 6000, True), ("f16", 300, 65, 9001, False),
         ("bf16", 1, 2048, 131001, True), ("bf16", 1024, 1024, 53000, True),
         ("bf16", 3000, 513, 45001, False), ("bf16", 16384, 1040, 4100, True)]


@pytest.mark.parametrize("smooth,c", [(0.0, 0.0), (0.1, 1e-3)])
@pytest.mark.parametrize("dtype,T,K,V,trans", CASES)
def test_dloss_keeps_its_digits(dtype, T, K, V, trans, smooth, c):
    assert dtype == "f16" or (T + 256) * K * V >= BIG
    a, b, target, _ = operands(T, K, V, DTYPES[dtype], trans)
    if T > 1:
        target[::5] = -100
    kw = dict(trans_b=trans, label_smoothing=smooth, z_loss=c)
    _, lse = mt.linear_cross_entropy(a, b, target, **kw)
    da1, db1 = db_of(2.0 ** -10, a, b, target, lse, **kw)
    for value in (FACTOR, 1e3 * FACTOR, -FACTOR):
        da, db = db_of(value, a, b, target, lse, **kw)
        ratio = torch.tensor(value, device="cuda").double() * 2 ** 10
        off = (db.double() - ratio * db1.double()).norm() / (abs(ratio) * db1.double().norm())
        assert off < 2.0 ** -13, off
        # dA is rounded to 16 bits on both sides.
        step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
        if abs(value) < 1:
            off = (da.double() - ratio * da1.double()).norm() / (abs(ratio) * da1.double().norm())
            assert off < 2 * step


@pytest.mark.parametrize("dtype,T,K,V,trans", CASES)
@pytest.mark.parametrize("sizes", ["equal", "random", "wide", "one", "none", "not finite"])
def test_against_64_bits(monkeypatch, dtype, T, K, V, trans, sizes):
    """Losses of all kinds that decide the scale.  The smallest of "wide", some 1e-34,
    give values of dA below 2^-126, where bf16's steps are 2^-133 however small the
    value: half a step, 2^-134 = 4.6e-41, more for what is stored in bf16."""
    of_normal = loss_tests.stored_step
    monkeypatch.setattr(loss_tests, "stored_step", lambda want, dt: of_normal(want, dt) + (
        2.0 ** -134 if dt == torch.bfloat16 else 0.0))
    a, b, target, dloss = operands(T, K, V, DTYPES[dtype], trans)
    if T > 2:
        target[1::3] = -100
    if sizes == "equal":
        dloss[:] = -1 / 1021
    elif sizes == "wide":
        dloss *= torch.logspace(-30, 0, T, device="cuda")
    elif sizes == "one":
        dloss[1:] = 0.0
    elif sizes == "none":
        dloss[:] = 0.0
    elif sizes == "not finite":
        dloss[1::3] = torch.tensor([float("nan"), float("inf"), 1e38],
                                   device="cuda").repeat(T)[:len(dloss[1::3])]
    check_grad(a, b, target, dloss, trans, 0.1, 1e-3, db_dtype=torch.float32)
