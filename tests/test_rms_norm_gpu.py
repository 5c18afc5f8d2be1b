"""GPU: mt_rms_norm (rms_norm) against the definition in 64 bits.

Tolerances (u = 2^-24 of fp32, s = 2^-11, 2^-8 or u of the storage type):
* r: the sum of d squares is added pairwise over threads and at most 64 deep
  within one, the reciprocal root is good to 2 ulp: (64 + 16) u / 2 + 4 u of
  r, taken as 64 u.
* h: one fp32 addition and one rounding: (s + 2 u) |h|.
* y: h, r and weight each good to the above: one rounding s plus 70 u, of
  |y|; subnormal results of fp16 round to a grid of 2^-24: half of it more.
* scale: 70 u of it.  q: q * scale is within half an e4m3 step of y (2^-4 of
  |y|, or half of the subnormal step 2^-9 of the scale) plus 80 u * 448 * scale
  for y and the scale's own rounding.
"""
import numpy as np
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: U}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


def rows_of(g, rows, d, pitch, dt, scale=1.0):
    """rows x d values in a rows x pitch buffer whose other columns are NaN."""
    buf = torch.full((rows, pitch), float("nan"), dtype=dt)
    buf[:, :d] = (torch.randn(rows, d, generator=g) * scale).to(dt)
    return buf.cuda()[:, :d]


def definition(x, res, weight, eps):
    h = x.double() + (res.double() if res is not None else 0)
    mean = (h * h).sum(1) / max(x.shape[1], 1)
    r = 1 / torch.sqrt(mean + eps)
    y = h * r[:, None]
    return h, r, y * weight.double() if weight is not None else y


def within(got, want, bound):
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"max excess {((got - want).abs() - bound).max().item():.3g}"


def check(x, res, weight, eps, out_dtype=None, **kw):
    dt = x.dtype
    got = mt.rms_norm(x, weight, residual=res, eps=eps, out_dtype=out_dtype, **kw)
    h, r, y = definition(x, res, weight, eps)
    s = STEP[dt]
    tiny = 2.0 ** -25 if dt == torch.float16 else 2.0 ** -150
    if out_dtype is None:
        yg, hg, rg = got
        assert yg.dtype == dt and yg.shape == x.shape
        within(yg, y, (s + 70 * U) * y.abs() + tiny)
    else:
        q, scale, hg, rg = got
        assert q.dtype == E4M3 and scale.dtype == torch.float32 and scale.shape == (x.shape[0],)
        want = torch.clamp(y.abs().amax(1) / 448, min=mt.MT_SCALE_MIN)
        within(scale, want, 70 * U * want)
        sc = scale.double()[:, None]
        within(q.float().double() * sc, y,
               torch.maximum(y.abs() * 2.0 ** -4, sc * 2.0 ** -10) + 80 * U * 448 * sc)
        assert (q.float().abs() <= 448).all()
    within(rg, r, 64 * U * r)
    if res is None:
        assert hg is x
    else:
        within(hg, h, (s + 2 * U) * h.abs() + tiny)


@pytest.mark.parametrize("dt", sorted(DTYPES))
@pytest.mark.parametrize("out", ["same", "e4m3"])
@pytest.mark.parametrize("rows,d,pad", [(1, 1, 0), (1, 4096, 0), (3, 7, 2), (37, 64, 0),
                                        (5, 255, 1), (9, 1000, 24), (130, 1024, 0),
                                        (2, 2056, 3), (17, 3001, 0), (4, 5120, 8), (3, 8191, 0),
                                        (6, 8192, 0), (2, 16384, 0), (2, 16392, 0),
                                        (2, 40001, 0)])
@pytest.mark.parametrize("residual", [False, True])
def test_matches_the_definition(dt, out, rows, d, pad, residual):
    g = torch.Generator().manual_seed(rows * 100003 + d)
    t = DTYPES[dt]
    x = rows_of(g, rows, d, d + pad, t)
    res = rows_of(g, rows, d, d + 2 * pad, t, 3.0) if residual else None
    w = (1 + 0.25 * torch.randn(d, generator=g)).cuda()
    if rows % 2:
        w = w.to(t)
    check(x, res, w, 1e-5, E4M3 if out == "e4m3" else None)


@pytest.mark.parametrize("d", [64, 1000, 4096, 20000])
def test_many_rows_no_weight(d):
    g = torch.Generator().manual_seed(d)
    check(rows_of(g, 1500, d, d, torch.bfloat16), None, None, 0.0)


@pytest.mark.parametrize("out_dtype", [None, E4M3])
@pytest.mark.parametrize("d", [48, 1001, 4096, 17000])
def test_rows_of_zeros_and_of_extremes(d, out_dtype):
    """Zeros (eps alone decides r), the type's smallest and largest values."""
    x = torch.zeros(4, d, dtype=torch.float16, device="cuda")
    x[1] = 2.0 ** -24
    x[2] = 65504.0
    x[3, d // 2] = -65504.0
    check(x, None, torch.ones(d, device="cuda"), 1e-6, out_dtype)
    got = mt.rms_norm(x, None, eps=1e-6, out_dtype=out_dtype)
    assert (got[0][0].float() == 0).all()
    if out_dtype is not None:
        assert got[1][0].item() == mt.MT_SCALE_MIN


@pytest.mark.parametrize("d", [40, 4096, 4097, 20000])
def test_nan_and_infinity_stay_in_their_rows(d):
    x = torch.ones(5, d, dtype=torch.bfloat16, device="cuda")
    x[1, d - 1] = float("nan")
    x[3, 0] = float("inf")
    y, _, r = mt.rms_norm(x, None, eps=0.0)
    assert torch.isnan(y[1].float()).all() and torch.isnan(r[1])
    assert r[3].item() == 0 and torch.isnan(y[3, 0]) and (y[3, 1:].float() == 0).all()
    for i in (0, 2, 4):
        assert (y[i].float() == 1).all() and r[i].item() == 1
    q, scale, _, r8 = mt.rms_norm(x, None, eps=0.0, out_dtype=E4M3)
    assert torch.equal(r8.isnan(), r.isnan())
    for i in (1, 3):
        assert torch.isnan(q[i].float()).all() and torch.isnan(scale[i])
    for i in (0, 2, 4):
        assert (q[i].float() == 448).all()


@pytest.mark.parametrize("d", [96, 1001, 8192, 20000])
def test_in_place_residual_and_given_outputs(d):
    g = torch.Generator().manual_seed(5)
    x, res = rows_of(g, 33, d, d, torch.bfloat16), rows_of(g, 33, d, d, torch.bfloat16)
    w = torch.randn(d, generator=g).cuda()
    y0, h0, r0 = mt.rms_norm(x, w, residual=res)
    xs, rs = x.clone(), res.clone()
    y1, h1, r1 = mt.rms_norm(xs, w, residual=rs, out=xs, h_out=rs)
    assert y1 is xs and h1 is rs
    assert torch.equal(y0, y1) and torch.equal(h0, h1) and torch.equal(r0, r1)


def test_empty():
    y, h, r = mt.rms_norm(torch.empty(0, 64, device="cuda"), None)
    assert y.shape == (0, 64) and r.shape == (0,)
    y, h, r = mt.rms_norm(torch.empty(3, 0, device="cuda"), None, eps=0.25)
    assert y.shape == (3, 0) and (r == 2).all()


def test_on_another_stream_and_from_a_graph():
    g = torch.Generator().manual_seed(9)
    x, w = rows_of(g, 64, 4096, 4096, torch.float16), torch.ones(4096, device="cuda")
    want = mt.rms_norm(x, w)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = mt.rms_norm(x, w)[0]
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = mt.rms_norm(x, w)[0]
    x.neg_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -want)


def test_refusals():
    x = torch.zeros(4, 8, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(8, device="cuda")
    with pytest.raises(TypeError):
        mt.rms_norm(x.cpu(), w)
    with pytest.raises(TypeError):
        mt.rms_norm(x.double(), w)
    with pytest.raises(TypeError):
        mt.rms_norm(x, w.half())
    with pytest.raises(TypeError):
        mt.rms_norm(x, w, residual=x.half())
    with pytest.raises(TypeError):
        mt.rms_norm(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mt.rms_norm(x, w[:4])
    with pytest.raises(ValueError):
        mt.rms_norm(x, w, residual=x[:2])
    with pytest.raises(ValueError):
        mt.rms_norm(x.t(), w[:4])
    with pytest.raises(ValueError):
        mt.rms_norm(x, w, h_out=x)
    with pytest.raises(mt.MtError) as e:
        mt.rms_norm(x, w, eps=-1.0)
    assert e.value.status == mt.MT_ERR_INVALID_ARG
    with pytest.raises(mt.MtError) as e:
        mt.rms_norm(x, w, residual=x.clone(), h_out=torch.zeros(5, 8, device="cuda",
                    dtype=torch.bfloat16)[1:], out=x[:, :].view(4, 8).as_strided((4, 8), (8, 1)),
                    eps=float("nan"))
    assert e.value.status == mt.MT_ERR_INVALID_ARG
    buf = torch.zeros(6, 8, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(mt.MtError) as e:
        mt.rms_norm(buf[:4], w, out=buf[1:5])
    assert e.value.status == mt.MT_ERR_ALIAS
