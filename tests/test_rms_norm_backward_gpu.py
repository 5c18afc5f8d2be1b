"""GPU: mt_rms_norm_backward against its formula in 64 bits, and the formula
against differences of the norm's own definition.

Tolerances (u = 2^-24, s: half a step of the storage type): the mean of d
products is added at most 64 deep in one thread, then over threads, each
product good to 4 u: 80 u of the mean of their absolute values, A.  dx is
then within s |dx| + 8 u (|terms|) + 80 u * r * |xhat| * A.  dweight adds one
product per row, at most rows / 8 deep in one thread: its bound is
(8 + 2 * depth) u of the sum of absolute values, with depth 300 for the sizes
here.
"""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: U}


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


def rows_of(g, rows, d, pitch, dt, scale=1.0):
    buf = torch.full((rows, pitch), float("nan"), dtype=dt)
    buf[:, :d] = (torch.randn(rows, d, generator=g) * scale).to(dt)
    return buf.cuda()[:, :d]


def formula(dy, h, w, r, dh):
    dy, h, r = dy.double(), h.double(), r.double()[:, None]
    w = torch.ones(dy.shape[1], dtype=torch.float64, device=dy.device) if w is None \
        else w.double()
    xhat, g = h * r, dy * w
    prod = g * xhat
    d = max(dy.shape[1], 1)
    dx = r * (g - xhat * (prod.sum(1, keepdim=True) / d))
    spread = r * xhat.abs() * (prod.abs().sum(1, keepdim=True) / d)
    size = (r * g).abs() + spread
    if dh is not None:
        dx = dx + dh.double()
        size = size + dh.double().abs()
    terms = dy * xhat
    return dx, size, spread, terms.sum(0), terms.abs().sum(0)


def check(dy, h, w, r, dh, **kw):
    dx, size, spread, dw, dw_abs = formula(dy, h, w, r, dh)
    got, got_w = mt.rms_norm_backward(dy, h, w, r, dh=dh, **kw)
    s = STEP[dy.dtype]
    tiny = 2.0 ** -25 if dy.dtype == torch.float16 else 2.0 ** -140
    assert got.dtype == dy.dtype and got_w.dtype == torch.float32
    err = (got.double() - dx).abs()
    assert (err <= s * dx.abs() + 8 * U * size + 80 * U * spread + tiny).all()
    err = (got_w.double() - dw).abs()
    assert (err <= 608 * U * dw_abs + 1e-40).all()
    return got, got_w


@pytest.mark.parametrize("dt", sorted(DTYPES))
@pytest.mark.parametrize("rows,d,pad", [(1, 1, 0), (1, 4096, 0), (3, 7, 2), (37, 64, 0),
                                        (5, 255, 1), (130, 1024, 0), (500, 2056, 3),
                                        (2053, 3001, 0), (64, 5120, 8), (3, 8191, 0),
                                        (700, 8192, 0), (33, 16384, 0), (2, 16392, 0),
                                        (40, 40001, 0)])
@pytest.mark.parametrize("carried", [False, True])
def test_matches_the_formula(dt, rows, d, pad, carried):
    g = torch.Generator().manual_seed(rows * 70001 + d)
    t = DTYPES[dt]
    dy, h = rows_of(g, rows, d, d + pad, t), rows_of(g, rows, d, d + 2 * pad, t, 2.0)
    dh = rows_of(g, rows, d, d + pad, t) if carried else None
    w = (1 + 0.25 * torch.randn(d, generator=g)).cuda()
    if rows % 2:
        w = w.to(t)
    r = torch.rsqrt(h.double().square().mean(1) + 1e-5).float()
    check(dy, h, w, r, dh)


@pytest.mark.parametrize("d", [64, 999, 4096])
def test_many_rows_give_the_same_bits_each_time(d):
    g = torch.Generator().manual_seed(d)
    dy, h = rows_of(g, 4800, d, d, torch.bfloat16), rows_of(g, 4800, d, d, torch.bfloat16)
    r = torch.rsqrt(h.float().square().mean(1))
    first = check(dy, h, None, r, None)
    for _ in range(3):
        again = mt.rms_norm_backward(dy, h, None, r)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("d", [24, 1000])
def test_formula_against_differences(d):
    """The gradient of sum(y * dy) + sum(h * dh) by central differences of
    the definition in 64 bits, along random directions of x and weight."""
    g = torch.Generator().manual_seed(3 * d)
    h = torch.randn(6, d, generator=g).cuda()
    dy, dh = torch.randn(6, d, generator=g).cuda(), torch.randn(6, d, generator=g).cuda()
    w, eps = (1 + 0.25 * torch.randn(d, generator=g)).cuda(), 1e-3

    def f(x, wt):
        y = x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps) * wt
        return (y * dy.double()).sum() + (x * dh.double()).sum()

    _, _, r = mt.rms_norm(h, w, eps=eps)
    dx, dw = mt.rms_norm_backward(dy, h, w, r, dh=dh)
    for _ in range(4):
        u = torch.randn(6, d, generator=g, dtype=torch.float64).cuda()
        v = torch.randn(d, generator=g, dtype=torch.float64).cuda()
        t = 1e-4
        x0, w0 = h.double(), w.double()
        num = (f(x0 + t * u, w0 + t * v) - f(x0 - t * u, w0 - t * v)) / (2 * t)
        terms = torch.cat([(dx.double() * u).flatten(), dw.double() * v])
        # Differences: t^2 times third derivatives (below 100 of the size
        # here); the kernel: 200 u of the terms' size.
        assert abs(terms.sum() - num) <= (100 * t * t + 200 * U) * terms.abs().sum()


@pytest.mark.parametrize("d", [40, 4096, 20000])
def test_nan_stays_in_its_row(d):
    dy = torch.ones(5, d, dtype=torch.bfloat16, device="cuda")
    h = dy.clone()
    dy[2, d - 1] = float("nan")
    dx, dw = mt.rms_norm_backward(dy, h, None, torch.ones(5, device="cuda"))
    assert dx[2].isnan().all()
    for i in (0, 1, 3, 4):
        assert (dx[i].float() == 0).all()
    assert dw[d - 1].isnan() and (dw[:d - 1] == 5).all()


@pytest.mark.parametrize("d", [96, 1001, 8192, 20000])
@pytest.mark.parametrize("into", ["dy", "dh"])
def test_in_place(d, into):
    g = torch.Generator().manual_seed(5)
    dy, h, dh = (rows_of(g, 33, d, d, torch.float16) for _ in range(3))
    r = torch.rand(33, generator=g).cuda()
    w = torch.randn(d, generator=g).cuda()
    want = mt.rms_norm_backward(dy, h, w, r, dh=dh)
    got = mt.rms_norm_backward(dy, h, w, r, dh=dh, out=dy if into == "dy" else dh)
    assert got[0] is (dy if into == "dy" else dh)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_empty_and_without_weight_gradient():
    e = torch.empty(0, 64, device="cuda")
    dx, dw = mt.rms_norm_backward(e, e, None, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and (dw == 0).all()
    x = torch.ones(3, 64, device="cuda")
    dx, dw = mt.rms_norm_backward(x, x, None, torch.ones(3, device="cuda"), need_weight=False)
    assert dw is None and (dx == 0).all()


def test_refusals():
    x = torch.zeros(4, 8, device="cuda", dtype=torch.bfloat16)
    r = torch.ones(4, device="cuda")
    with pytest.raises(TypeError):
        mt.rms_norm_backward(x, x.half(), None, r)
    with pytest.raises(TypeError):
        mt.rms_norm_backward(x, x, None, r.half())
    with pytest.raises(ValueError):
        mt.rms_norm_backward(x, x, None, r[:3])
    with pytest.raises(ValueError):
        mt.rms_norm_backward(x, x[:, :4], None, r)
    with pytest.raises(mt.MtError) as e:
        mt.rms_norm_backward(x, x, None, r, out=x)   # dx may be dy, not h
    assert e.value.status == mt.MT_ERR_ALIAS
