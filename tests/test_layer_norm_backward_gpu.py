"""GPU: mt_layer_norm_backward against its formula in 64 bits, and the formula
against differences of the layer norm's definition.

Tolerances (u = 2^-24, s half a step of the storage type): with xhat = (h - m) r,
within 2 u of itself, g = dy w within u, and sums of a row at most N = 48 + d / 512
deep, dres is within
  u r (6 |g| + (N + 6) mean|g| + |xhat| (N + 10) mean|g xhat|) + 4 u (|dres| + |dh|)
plus its rounding s |dres|; dx = D(dres) is that over 1 - p (2 u more) plus its own
rounding.  A column's sum over the rows is at most rows / 8 + 64 deep.
"""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from test_layer_norm_gpu import (DTYPES, STEP, U, mask_by_columns, rows_of, seed_of, stored_step,
                                 within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


def formula(dy, h, w, mean, rstd, dh):
    dy, xh = dy.double(), (h.double() - mean.double()[:, None]) * rstd.double()[:, None]
    r = rstd.double()[:, None]
    g = dy * w.double() if w is not None else dy
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dres = r * (g - c1 - xh * c2)
    if dh is not None:
        dres = dres + dh.double()
    n = 48 + h.shape[1] / 512
    bound = U * r * (6 * g.abs() + (n + 6) * g.abs().mean(1, keepdim=True)
                     + xh.abs() * (n + 10) * (g * xh).abs().mean(1, keepdim=True)) + \
        4 * U * (dres.abs() + (dh.double().abs() if dh is not None else 0.0))
    return dres, bound, dy * xh, dy


def statistics(h, eps=1e-5):
    h = h.float()
    mean = h.mean(1)
    return mean, ((h - mean[:, None]).square().mean(1) + eps).rsqrt()


def check(dy, h, w, dh, p=0.0, seed=0, sequence=0, **kw):
    rows, d = h.shape
    dt = h.dtype
    mean, rstd = statistics(h)
    dres, bound, pw, pb = formula(dy, h, w, mean, rstd, dh)
    got = mt.layer_norm_backward(dy, h, w, mean, rstd, dh=dh, dropout=p, seed=seed_of(seed),
                                 sequence=sequence, **kw)
    within(got[1], dres, bound + stored_step(dres, dt) + STEP[dt] * bound)
    if p:
        keep = mask_by_columns(rows, d, p, seed, sequence)
        dx, e = torch.where(keep, dres, 0.0) / (1 - p), bound / (1 - p)
        within(got[0], dx, e + 3 * U * dx.abs() + stored_step(dx, dt) + STEP[dt] * e)
        assert not got[0][~keep].any()
    else:
        assert got[0] is got[1]
    depth = (rows / 8 + 64 + 4) * U
    for out, terms in ((got[2], pw), (got[3], pb)):
        if out is not None:
            within(out, terms.sum(0), depth * terms.abs().sum(0))
    return got


SIZES = [(1, 1), (2, 7), (3, 8), (5, 33), (4, 255), (9, 256), (3, 264), (700, 264), (2, 1000),
         (6, 1024), (5, 1025), (153, 2048), (3, 3001), (310, 3001), (200, 4096), (4, 5120),
         (155, 8192), (2, 8200), (3, 12288), (2, 16384), (2, 16392), (40, 20001)]


@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,d", SIZES)
def test_sizes(rows, d, dtype, p):
    g = torch.Generator().manual_seed(rows * 100003 + d)
    dt = DTYPES[dtype]
    for pad, other in ((0, False), (8, True), (3, True)):
        dy, h = rows_of(g, rows, d, d + pad, dt, 0.5), rows_of(g, rows, d, d + pad, dt, 2.0, 0.3)
        dh = rows_of(g, rows, d, d + pad, dt, 0.5)
        w = (1 + 0.1 * torch.randn(d, generator=g)).cuda().to(torch.float32 if other else dt)
        check(dy, h, w, dh if other else None, p, 5 + d, 3)
    check(dy, h, None, None, p, -d, 2 ** 50, need_weight=rows % 2 == 0, need_bias=rows % 2 == 1)


@pytest.mark.parametrize("d", [64, 250, 4096, 20000])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_in_place(d, p):
    g = torch.Generator().manual_seed(d)
    dy, h, dh = (rows_of(g, 300, d, d, torch.bfloat16) for _ in range(3))
    mean, rstd = statistics(h)
    kw = dict(dropout=p, seed=seed_of(5), sequence=1)
    want = mt.layer_norm_backward(dy, h, None, mean, rstd, dh=dh, **kw)
    for which in (0, 1):
        a, b = dy.clone(), dh.clone()
        got = mt.layer_norm_backward(a, h, None, mean, rstd, dh=b, out=(a, b)[which], **kw)
        assert got[0] is (a, b)[which]
        for u, v in zip(got, want):
            assert torch.equal(u, v)


@pytest.mark.parametrize("d", [64, 3001, 4096])
def test_same_bits_every_time(d):
    g = torch.Generator().manual_seed(d)
    dy, h = (rows_of(g, 1000, d, d, torch.bfloat16) for _ in range(2))
    mean, rstd = statistics(h)
    first = mt.layer_norm_backward(dy, h, None, mean, rstd)
    for _ in range(3):
        for a, b in zip(first, mt.layer_norm_backward(dy, h, None, mean, rstd)):
            assert torch.equal(a, b)


def test_no_rows_and_no_columns():
    e = torch.empty(0, device="cuda")
    dx, dres, dw, db = mt.layer_norm_backward(torch.empty(0, 24, device="cuda"),
                                              torch.empty(0, 24, device="cuda"), None, e, e)
    assert dx.shape == (0, 24)
    assert torch.equal(dw.cpu(), torch.zeros(24)) and torch.equal(db.cpu(), torch.zeros(24))
    z = torch.zeros(3, device="cuda")
    assert mt.layer_norm_backward(torch.empty(3, 0, device="cuda"), torch.empty(3, 0, device="cuda"),
                                  None, z, z)[2].shape == (0,)


def test_rows_of_zero_rstd_pass_the_streams_gradient_alone():
    h = torch.full((2, 512), 3.0, device="cuda")
    dy, dh = torch.randn(2, 512, device="cuda"), torch.randn(2, 512, device="cuda")
    _, _, mean, rstd = mt.layer_norm(h, eps=0.0)
    assert not rstd.any()
    assert torch.equal(mt.layer_norm_backward(dy, h, None, mean, rstd, dh=dh)[0], dh)


def test_formula_against_differences():
    """Central differences of the definition in 64 bits, along random
    directions of x, residual, weight and bias; steps of 1e-5 leave 1e-9 of the
    scale of a gradient."""
    g = torch.Generator().manual_seed(1)
    draw = lambda *s: torch.randn(*s, generator=g).double().cuda()  # noqa: E731
    rows, d, p = 6, 40, 0.25
    x, res, w, b, dy, dh = draw(rows, d), draw(rows, d), draw(d), draw(d), draw(rows, d), draw(rows, d)
    keep = mask_by_columns(rows, d, p, 9, 4)

    def objective(x, res, w, b):
        h = torch.where(keep, x / (1 - p), 0.0) + res
        m = h.mean(1, keepdim=True)
        r = ((h - m).square().mean(1, keepdim=True) + 1e-5).rsqrt()
        return (((h - m) * r * w + b) * dy).sum() + (h * dh).sum()

    h = torch.where(keep, x / (1 - p), 0.0) + res
    mean = h.mean(1)
    rstd = ((h - mean[:, None]).square().mean(1) + 1e-5).rsqrt()
    dres, _, pw, pb = formula(dy, h, w, mean, rstd, dh)
    grads = torch.where(keep, dres / (1 - p), 0.0), dres, pw.sum(0), pb.sum(0)
    at = [x, res, w, b]
    for i, grad in enumerate(grads):
        v = draw(*grad.shape)
        step = 1e-5
        up = objective(*[t + step * v if k == i else t for k, t in enumerate(at)])
        down = objective(*[t - step * v if k == i else t for k, t in enumerate(at)])
        assert abs((up - down) / (2 * step) - (grad * v).sum()) < 1e-6 * grad.norm() * v.norm()


@pytest.mark.parametrize("dt", [torch.float16, torch.float32])
def test_bounded_wait_runs_out(dt):
    """The staged rows' copies withheld: the waits run out, the call reports it,
    and the next call is right."""
    from tiled_fp32_gemm_gb300 import model
    g = torch.Generator().manual_seed(3)
    dy, h = rows_of(g, 40, 512, 512, dt), rows_of(g, 40, 512, 512, dt)
    mean, rstd = statistics(h)
    dx = torch.empty_like(dy)
    code = {torch.float16: 1, torch.float32: mt.MT_DTYPE_F32}[dt]
    a = model.mt_layer_norm_backward_args(
        rows=40, d=512, dy=dy.data_ptr(), lddy=512, h=h.data_ptr(), ldh=512, mean=mean.data_ptr(),
        rstd=rstd.data_ptr(), dx=dx.data_ptr(), lddx=512, dtype=code, fault_inject=1)
    stream = torch.cuda.current_stream().cuda_stream
    assert mt.mt_check_device_status(stream) == mt.MT_OK
    assert mt.mt_layer_norm_backward(a, stream) == mt.MT_OK
    assert mt.mt_check_device_status(stream) == mt.MT_ERR_TIMEOUT
    assert mt.mt_check_device_status(stream) == mt.MT_OK
    check(dy, h, None, None)
