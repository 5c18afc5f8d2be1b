"""GPU: mt_linear_cross_entropy and its gradient against their definitions in
64 bits, and the gradient's formula against differences.

Tolerances (u = 2^-24, s half a step of the storage type).  A logit's fp32 sum
is within e_z = 5e-5 |A| |B| of the exact one (the bar of the library's
tensor-core products; nothing where a row of A holds one value, whose products
are exact).  An exponential is good to 2^-22 and its argument to 2 u of the
logits' size, sums of positive terms to 64 u and the pieces' joins to 24 (2^-22):
lse is within max e_z + 2^-17 + 4 u (max|z| + |lse|).  The loss adds its
target's e_z and, with smoothing, the mean's: mean e_z + 512 u mean|z|.

D = g (p (1 + 2 c lse) - s_l / V - (1 - s_l) [target]) has p within p (e_z + E)
of itself, E = 2^-20 + 6 u (|z| + |lse|), and 6 u of each term more; it is rounded
to the storage type (fp16: held times a power of two that brings the largest
factor past 2^13, so its subnormal half step is 2^-38 of that factor).  The
products add 5e-5 of the sum of absolute values, results their own rounding.
"""
import math

import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from test_layer_norm_gpu import STEP, U, stored_step, within

pytestmark = pytest.mark.gpu

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
BAR = 5e-5


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


def stored(g, rows, cols, pad, dt, scale=1.0):
    """rows x cols values in a wider buffer whose other columns are NaN."""
    buf = torch.full((rows, cols + pad), float("nan"), device="cuda")
    buf[:, :cols] = torch.randn(rows, cols, generator=g, device="cuda") * scale
    return buf.to(dt)[:, :cols]


def operands(T, K, V, dt, trans, pad=0, seed=0, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed + 31 * T + 7 * K + V)
    a = stored(g, T, K, pad, dt)
    w = spread / math.sqrt(max(K, 1))
    b = stored(g, V, K, pad, dt, w) if trans else stored(g, K, V, pad, dt, w)
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    dloss = torch.randn(T, generator=g, device="cuda") / T
    return a, b, target, dloss


def logits(a, b, trans):
    """(z, e_z) in 64 bits."""
    A, W = a.double(), b.double().t() if trans else b.double()
    return A @ W, BAR * (A.abs() @ W.abs())


def check_loss(a, b, target, trans, smooth=0.0, c=0.0, ignore=-100, exact_sums=False, **kw):
    loss, lse = mt.linear_cross_entropy(a, b, target, trans_b=trans, ignore_index=ignore,
                                        label_smoothing=smooth, z_loss=c, **kw)
    z, ez = logits(a, b, trans)
    if exact_sums:
        ez = torch.zeros_like(ez)
    V = z.shape[1]
    want = torch.logsumexp(z, 1)
    el = ez.amax(1) + 2.0 ** -17 + 4 * U * (z.abs().amax(1) + want.abs())
    within(lse, want, el)
    live = target != ignore
    t = torch.where(live, target, 0)[:, None]
    zt, ezt = z.gather(1, t)[:, 0], ez.gather(1, t)[:, 0]
    value = want - (1 - smooth) * zt - smooth * z.mean(1) + c * want ** 2
    el = el * (1 + 2 * c * want.abs() + c * el) + ezt + 4 * U * (value.abs() + zt.abs())
    if smooth:
        el = el + ez.mean(1) + 512 * U * z.abs().mean(1) + 4 * U * zt.abs()
    within(loss[live], value[live], el[live])
    assert not loss[~live].any()
    return loss, lse


def check_grad(a, b, target, dloss, trans, smooth=0.0, c=0.0, ignore=-100, db_dtype=None,
               need=(True, True)):
    dt = a.dtype
    z, ez = logits(a, b, trans)
    V = z.shape[1]
    lse32 = torch.logsumexp(z, 1).float()
    lse = lse32.double()[:, None]
    da, db = mt.linear_cross_entropy_backward(
        dloss, a, b, target, lse32, trans_b=trans, ignore_index=ignore, label_smoothing=smooth,
        z_loss=c, need_a=need[0], need_b=need[1], db_dtype=db_dtype)
    live = target != ignore
    g = torch.where(live, dloss.double(), 0.0)[:, None]
    factor = 1 + 2 * c * lse
    p = (z - lse).exp() * factor
    hit = torch.zeros_like(z).scatter_(1, torch.where(live, target, 0)[:, None], 1 - smooth)
    D = g * (p - smooth / V - hit)
    E = ez + 2.0 ** -20 + 6 * U * (z.abs() + lse.abs())
    eD = g.abs() * (p.abs() * E * (1 + E) + 6 * U * (p.abs() + smooth / V + hit))
    if dt == torch.float16:
        eD = eD + 2.0 ** -38 * (g * factor).abs().amax() * live[:, None]
    eD = eD + STEP[dt] * (D.abs() + eD)
    A, W = a.double(), b.double() if trans else b.double().t()   # W: V x K
    if need[0]:
        want = D @ W
        e = eD @ W.abs() + BAR * (D.abs() + eD) @ W.abs()
        within(da, want, e + stored_step(want, dt) + STEP[dt] * e)
        assert not da[~live].any()
    else:
        assert da is None
    if need[1]:
        want = D.t() @ A
        e = eD.t() @ A.abs() + BAR * (D.abs() + eD).t() @ A.abs()
        if not trans:
            want, e = want.t(), e.t()
        out = db_dtype or dt
        assert db.dtype == out
        within(db, want, e + stored_step(want, out) + STEP[out] * e)
    else:
        assert db is None
    return da, db


# Few tokens (the split kernel, by its tile of tokens), pairs, edges of tiles
# of the vocabulary and of K.
SIZES = [(1, 8, 1), (1, 64, 2), (2, 65, 31), (3, 1, 33), (16, 200, 127), (17, 64, 128),
         (33, 63, 129), (64, 72, 257), (65, 130, 1000), (128, 64, 4099), (129, 64, 300),
         (255, 16, 7000), (256, 65, 8192), (257, 63, 5900), (513, 130, 4099), (1000, 64, 3001),
         (1, 1024, 20011), (30, 2048, 5000), (700, 257, 9000)]


@pytest.mark.parametrize("trans", [True, False])
@pytest.mark.parametrize("T,K,V", SIZES)
def test_sizes(T, K, V, trans):
    dt = torch.float16 if (T + V) % 2 else torch.bfloat16
    for pad in (0, 3):
        a, b, target, dloss = operands(T, K, V, dt, trans, pad)
        check_loss(a, b, target, trans)
        check_grad(a, b, target, dloss, trans)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("smooth,c", [(0.1, 0.0), (1.0, 0.0), (0.0, 1e-3), (0.3, 0.05)])
@pytest.mark.parametrize("T,K,V", [(5, 40, 300), (64, 64, 1001), (300, 72, 6000)])
def test_smoothing_and_z_loss(T, K, V, smooth, c, dtype):
    a, b, target, dloss = operands(T, K, V, DTYPES[dtype], True)
    target[::3] = -100
    check_loss(a, b, target, True, smooth, c)
    check_grad(a, b, target, dloss, True, smooth, c)
    check_grad(a, b, target, dloss, True, smooth, c, db_dtype=torch.float32)


@pytest.mark.parametrize("T,V", [(4, 700), (40, 900), (300, 6000)])
def test_exact_logits(T, V):
    """Rows of A with one value of 1: the logits are B's values, exactly, and
    lse and loss have to be good to the softmax's own error.  Large logits, a
    target far above the rest and equal logits among them."""
    K = 64
    a = torch.zeros(T, K, device="cuda", dtype=torch.bfloat16)
    a[torch.arange(T), torch.arange(T) % K] = 1.0
    b = operands(1, K, V, torch.bfloat16, True, spread=40.0)[1].clone()
    target = torch.arange(T, device="cuda") * 7 % V
    b[:, 0] = 3.0
    b[:, 1] = -100.0
    b[target[1], 1] = 100.0
    b[:, 2] = 20000.0
    b[:, 3] *= 30.0
    check_loss(a, b, target, True, exact_sums=True)
    check_loss(a, b, target, True, smooth=0.2, c=1e-4, exact_sums=True)
    loss, lse = mt.linear_cross_entropy(a, b, target, trans_b=True)
    assert abs(lse[0].item() - 3.0 - math.log(V)) <= 2.0 ** -17


def test_many_pieces_join_without_drift():
    """Equal logits over a large vocabulary: every join has the same maximum,
    and none may lose a digit of the sum."""
    V = 131071
    for T in (1, 300):
        a = torch.ones(T, 8, device="cuda", dtype=torch.bfloat16)
        b = torch.full((V, 8), 2.4375, device="cuda", dtype=torch.bfloat16)
        loss, lse = mt.linear_cross_entropy(a, b, torch.zeros(T, dtype=torch.int64, device="cuda"),
                                            trans_b=True)
        assert (lse.double() - 19.5 - math.log(V)).abs().max() < 2.0 ** -18
        assert (loss.double() - math.log(V)).abs().max() < 2.0 ** -18


@pytest.mark.parametrize("T", [1, 20, 200, 400])
@pytest.mark.parametrize("ignore", [-100, 0, 5])
def test_tokens_without_a_target(T, ignore):
    a, b, target, dloss = operands(T, 64, 6000, torch.bfloat16, True)
    target[torch.arange(T, device="cuda") % 3 != 1] = ignore
    check_loss(a, b, target, True, ignore=ignore)
    check_grad(a, b, target, dloss, True, ignore=ignore)
    target[:] = ignore
    loss, lse = check_loss(a, b, target, True, ignore=ignore)
    da, db = mt.linear_cross_entropy_backward(dloss, a, b, target, lse, trans_b=True,
                                              ignore_index=ignore)
    assert not da.any() and not db.any()


@pytest.mark.parametrize("T", [3, 300])
def test_ignored_rows_are_zeros_whatever_their_logits(T):
    """Padded tokens whose logits are NaN or infinite (their row of B's
    gradient's sums is finite: A's row is)."""
    a, b, target, dloss = operands(T, 64, 6000, torch.float16, True)
    target[1] = -100
    _, lse = mt.linear_cross_entropy(a, b, target, trans_b=True)
    lse[1] = float("nan")
    dloss[1] = float("inf")
    da, db = mt.linear_cross_entropy_backward(dloss, a, b, target, lse, trans_b=True)
    assert not da[1].any() and db.isfinite().all() and da.isfinite().all()


@pytest.mark.parametrize("T", [3, 300])
@pytest.mark.parametrize("bad", [-1, -2, 6000, 2 ** 40, -2 ** 63])
def test_targets_outside_the_vocabulary_are_nan(T, bad):
    a, b, target, dloss = operands(T, 64, 6000, torch.bfloat16, True)
    want, lse = mt.linear_cross_entropy(a, b, target, trans_b=True)
    target[1] = bad
    loss, lse = mt.linear_cross_entropy(a, b, target, trans_b=True)
    assert loss[1].isnan() and lse.isfinite().all()
    assert torch.equal(loss[2:], want[2:]) and torch.equal(loss[:1], want[:1])
    da, db = mt.linear_cross_entropy_backward(dloss, a, b, target, lse, trans_b=True)
    assert da[1].isnan().all() and da[2:].isfinite().all() and db.isnan().all()


@pytest.mark.parametrize("T", [2, 300])
def test_nan_logits_keep_to_their_token(T):
    a, b, target, _ = operands(T, 64, 6000, torch.bfloat16, True)
    want, _ = mt.linear_cross_entropy(a, b, target, trans_b=True)
    a[1, 5] = float("nan")
    loss, lse = mt.linear_cross_entropy(a, b, target, trans_b=True)
    assert loss[1].isnan() and lse[1].isnan()
    assert torch.equal(loss[2:], want[2:]) and torch.equal(loss[:1], want[:1])


@pytest.mark.parametrize("T", [1, 5, 200])
def test_no_contraction(T):
    """K = 0: logits of zeros."""
    a = torch.empty(T, 0, device="cuda", dtype=torch.bfloat16)
    b = torch.empty(3000, 0, device="cuda", dtype=torch.bfloat16)
    target = torch.zeros(T, dtype=torch.int64, device="cuda")
    loss, lse = mt.linear_cross_entropy(a, b, target, trans_b=True)
    assert (loss.double() - math.log(3000)).abs().max() < 2.0 ** -19
    da, db = mt.linear_cross_entropy_backward(loss, a, b, target, lse, trans_b=True)
    assert da.shape == (T, 0) and db.shape == (3000, 0)


@pytest.mark.parametrize("trans", [True, False])
def test_no_tokens(trans):
    a = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    b = operands(1, 64, 300, torch.bfloat16, trans)[1]
    none, zero = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = mt.linear_cross_entropy(a, b, zero, trans_b=trans)
    assert loss.shape == lse.shape == (0,)
    da, db = mt.linear_cross_entropy_backward(none, a, b, zero, none, trans_b=trans,
                                              db_dtype=torch.float32)
    assert da.shape == (0, 64) and db.shape == b.shape and not db.any()


@pytest.mark.parametrize("need", [(True, False), (False, True)])
@pytest.mark.parametrize("T,K,V", [(20, 64, 500), (700, 130, 9000)])
def test_one_gradient_alone_has_the_same_bits(T, K, V, need):
    a, b, target, dloss = operands(T, K, V, torch.float16, False)
    both = check_grad(a, b, target, dloss, False)
    one = check_grad(a, b, target, dloss, False, need=need)
    for x, y in zip(both, one):
        assert y is None or torch.equal(x, y)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("db_dtype", [None, torch.float32])
@pytest.mark.parametrize("T,K,V,trans", [(200, 1024, 9000, True), (30, 520, 20000, True),
                                         (300, 1040, 9008, False), (2000, 2048, 9100, True)])
def test_weight_gradients_on_pairs(T, K, V, trans, db_dtype, dtype):
    """Results that leave by boxes, 16- and 32-bit, with and without D's scale,
    ragged in rows and columns."""
    a, b, target, dloss = operands(T, K, V, DTYPES[dtype], trans)
    check_grad(a, b, target, dloss, trans, db_dtype=db_dtype)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("trans", [True, False])
@pytest.mark.parametrize("T,K,V", [(4096, 40, 40000), (8192, 64, 33001), (16384, 40, 40000),
                                   (20000, 66, 33001)])
def test_several_pieces_of_the_vocabulary(T, K, V, trans, dtype):
    a, b, target, dloss = operands(T, K, V, DTYPES[dtype], trans)
    check_grad(a, b, target, dloss, trans, smooth=0.1)


@pytest.mark.parametrize("size", [1e-30, 1e-6, 1.0, 1e4])
def test_fp16_gradients_keep_small_probabilities(size):
    """Losses scaled far up or down: D's scale follows them.  db in fp32 shows
    it (its own type does not round to zero)."""
    a, b, target, dloss = operands(300, 64, 6000, torch.float16, True)
    _, db = check_grad(a, b, target, dloss * size, True, db_dtype=torch.float32,
                       need=(size < 1e3, True))
    assert (db != 0).float().mean() > 0.99


@pytest.mark.parametrize("trans", [True, False])
@pytest.mark.parametrize("T,K,V", [(17, 64, 500), (700, 130, 9000)])
def test_same_bits_every_time(T, K, V, trans):
    a, b, target, dloss = operands(T, K, V, torch.bfloat16, trans)
    loss, lse = mt.linear_cross_entropy(a, b, target, trans_b=trans, label_smoothing=0.1)
    grads = mt.linear_cross_entropy_backward(dloss, a, b, target, lse, trans_b=trans)
    for _ in range(3):
        again = mt.linear_cross_entropy(a, b, target, trans_b=trans, label_smoothing=0.1)
        assert torch.equal(loss, again[0]) and torch.equal(lse, again[1])
        again = mt.linear_cross_entropy_backward(dloss, a, b, target, lse, trans_b=trans)
        assert all(torch.equal(x, y) for x, y in zip(grads, again))


def test_formula_against_differences():
    """Central differences of the loss in 64 bits along random directions."""
    g = torch.Generator().manual_seed(2)
    draw = lambda *s: torch.randn(*s, generator=g).double().cuda()  # noqa: E731
    T, K, V, s, c = 7, 12, 30, 0.2, 0.03
    a, w, dloss = draw(T, K), draw(V, K), draw(T)
    target = torch.arange(T, device="cuda") * 3

    def objective(a, w):
        z = a @ w.t()
        lse = torch.logsumexp(z, 1)
        loss = lse - (1 - s) * z.gather(1, target[:, None])[:, 0] - s * z.mean(1) + c * lse ** 2
        return (loss * dloss).sum()

    z = a @ w.t()
    lse = torch.logsumexp(z, 1)[:, None]
    hit = torch.zeros_like(z).scatter_(1, target[:, None], 1 - s)
    D = dloss[:, None] * ((z - lse).exp() * (1 + 2 * c * lse) - s / V - hit)
    for i, grad in enumerate((D @ w, D.t() @ a)):
        v, step = draw(*grad.shape), 1e-5
        at = [a, w]
        ends = [objective(*[t + k * step * v if j == i else t for j, t in enumerate(at)])
                for k in (1, -1)]
        assert abs((ends[0] - ends[1]) / (2 * step) - (grad * v).sum()) < \
            1e-6 * grad.norm() * v.norm()


@pytest.mark.parametrize("T", [4, 300])
def test_bounded_wait_runs_out(T):
    """The copies withheld: the waits run out, the call reports it, and the next
    call is right."""
    from tiled_fp32_gemm_gb300 import model
    a, b, target, _ = operands(T, 64, 6000, torch.bfloat16, True)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    args = model.mt_linear_cross_entropy_args(
        T=T, K=64, V=6000, A=a.data_ptr(), lda=64, B=b.data_ptr(), ldb=64,
        target=target.data_ptr(), loss=loss.data_ptr(), lse=lse.data_ptr(), ignore_index=-100,
        trans_b=1, dtype=2, fault_inject=1)
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    assert mt.mt_check_device_status(stream) == mt.MT_OK
    assert mt.mt_linear_cross_entropy(args, stream) == mt.MT_OK
    assert mt.mt_check_device_status(stream) == mt.MT_ERR_TIMEOUT
    assert mt.mt_check_device_status(stream) == mt.MT_OK
    check_loss(a, b, target, True)
