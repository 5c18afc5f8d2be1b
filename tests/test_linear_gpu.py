"""GPU: mt_linear (linear) against the definition in 64 bits.

Tolerance: the product's fp32 sums are within 5e-5 * W of the exact ones, W =
|A| * |B| (the bar of the library's tensor-core products), scaled by the two
scales; the bias adds one rounding.  The activations' slopes are below 1.13
and their fp32 evaluation is good to 8 ulp of |z|; residual and storage round
once each.
"""
import numpy as np
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: U}
E4M3 = torch.float8_e4m3fn
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


def stored(g, rows, cols, pitch, dt, scale=1.0):
    """rows x cols values in a rows x pitch buffer whose other columns are NaN."""
    buf = torch.full((rows, pitch), float("nan"))
    buf[:, :cols] = torch.randn(rows, cols, generator=g) * scale
    return buf.to(dt).cuda()[:, :cols]


def act64(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / 2 ** 0.5)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def check(a, b, bias=None, act="none", res=None, trans=False, sa=None, sb=None, out_dtype=None,
          preact=False):
    got = mt.linear(a, b, bias=bias, activation=act, residual=res, trans_b=trans, scale_a=sa,
                    scale_b=sb, out_dtype=out_dtype, preact=preact)
    assert mt.mt_check_device_status(0) == mt.MT_OK
    y, z = got if preact else (got, None)
    A, B = a.float().double(), b.float().double()
    B = B.t() if trans else B
    P, W = A @ B, A.abs() @ B.abs()
    if sa is not None:
        s = sa.double()[:, None] * sb.double()
        P, W = P * s, W * s.abs()
    if bias is not None:
        P, W = P + bias.double(), W + bias.double().abs()
    dt = out_dtype or (torch.bfloat16 if a.dtype == E4M3 else a.dtype)
    s = STEP[dt]
    tiny = 2.0 ** -25 if dt == torch.float16 else 2.0 ** -130
    want = act64(P, act)
    tol = 1.13 * 5e-5 * W + 16 * U * P.abs()
    if res is not None:
        want = want + res.double()
        tol = tol + 2 * U * want.abs()
    assert y.dtype == dt and y.shape == want.shape
    err = (y.double() - want).abs()
    assert (err <= tol * (1 + s) + s * want.abs() + tiny).all(), (err - tol).max()
    if preact:
        err = (z.double() - P).abs()
        assert (err <= 5e-5 * W * (1 + s) + s * P.abs() + tiny).all()
    return got


SHAPES = [(1, 128, 64), (1, 1, 1), (1, 4096, 4096), (2, 1000, 777), (15, 129, 200),
          (16, 4096, 512), (17, 130, 130), (24, 640, 8192), (32, 333, 96), (33, 127, 65),
          (64, 512, 1024), (65, 200, 1000), (100, 72, 80), (128, 1024, 1024), (129, 257, 513),
          (300, 264, 1000), (1, 128, 40000), (513, 700, 24)]


@pytest.mark.parametrize("dt", sorted(DTYPES))
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_matches_the_definition(dt, trans, M, N, K, pad):
    g = torch.Generator().manual_seed(M + 7 * N + 13 * K + pad)
    t = DTYPES[dt]
    a = stored(g, M, K, K + pad, t)
    b = stored(g, *((N, K + pad) if trans else (K, N + pad)), (K if trans else N) + pad, t,
               K ** -0.5)
    b = b[:, :K] if trans else b[:, :N]
    bias = torch.randn(N, generator=g).cuda() if M % 2 else None
    res = stored(g, M, N, N + pad, t) if N % 2 else None
    check(a, b, bias, ACTS[(M + N + K) % 5], res, trans, preact=K % 2 == 0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out_dtype", [None, torch.float32])
@pytest.mark.parametrize("M", [1, 40, 200])
def test_every_activation_over_its_range(act, out_dtype, M):
    """Pre-activations from -120 to 120 (past the overflow of exp)."""
    g = torch.Generator().manual_seed(M)
    a = stored(g, M, 96, 96, torch.bfloat16)
    b = stored(g, 96, 256, 256, torch.bfloat16, 2.0)
    bias = torch.linspace(-60, 60, 256).cuda()
    res = stored(g, M, 256, 256, out_dtype or torch.bfloat16)
    check(a, b, bias, act, res, out_dtype=out_dtype, preact=True)


@pytest.mark.parametrize("M,N,K", SHAPES + [(700, 900, 640)])
@pytest.mark.parametrize("pad", [0, 16, 3])
@pytest.mark.parametrize("out", [None, torch.float16, torch.float32])
def test_8_bit(M, N, K, pad, out):
    g = torch.Generator().manual_seed(M + 5 * N + 11 * K + pad)
    a = stored(g, M, K, K + pad, E4M3, 40.0)
    b = stored(g, N, K, K, E4M3, 40.0)
    sa = (torch.rand(M, generator=g) + 0.5).cuda() / 40
    sb = (torch.rand(N, generator=g) + 0.5).cuda() / 40 * K ** -0.5
    bias = torch.randn(N, generator=g).cuda() if M % 2 else None
    res = stored(g, M, N, N + pad, out or torch.bfloat16) if N % 2 else None
    check(a, b, bias, ACTS[(M + N) % 5], res, True, sa, sb, out)


@pytest.mark.parametrize("dt", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("M,N,K,pad", [(2500, 2305, 640, 0), (2305, 2561, 77, 5),
                                       (1, 40000, 64, 0), (20000, 256, 128, 8)])
@pytest.mark.parametrize("out", [None, torch.float32])
def test_tiles_that_fill_the_gpu(dt, trans, M, N, K, pad, out):
    """Enough 256 x 256 tiles for the CTA-pair kernel, with ragged edges."""
    if dt == "e4m3" and not trans:
        return
    g = torch.Generator().manual_seed(M + N)
    t = E4M3 if dt == "e4m3" else DTYPES[dt]
    a = stored(g, M, K, K + pad, t)
    b = stored(g, *((N, K) if trans else (K, N)), (K if trans else N) + pad, t, K ** -0.5)
    res = stored(g, M, N, N + pad, out or (torch.bfloat16 if dt == "e4m3" else t))
    sa = sb = None
    if dt == "e4m3":
        sa, sb = torch.rand(M, generator=g).cuda() + 0.5, torch.rand(N, generator=g).cuda() + 0.5
    check(a, b, torch.randn(N, generator=g).cuda(), "gelu", res, trans, sa, sb, out,
          preact=K % 2 == 0)


@pytest.mark.parametrize("dt", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(3, 200, 4100), (130, 300, 1000), (600, 520, 256),
                                   (2304, 2304, 300)])
def test_integers_are_exact(dt, M, N, K):
    g = np.random.default_rng(M)
    t = E4M3 if dt == "e4m3" else DTYPES[dt]
    A = torch.from_numpy(g.integers(-8, 9, (M, K)).astype(np.float32))
    B = torch.from_numpy(g.integers(-8, 9, (N, K)).astype(np.float32))
    kw = {}
    if dt == "e4m3":
        kw = dict(scale_a=torch.full((M,), 2.0).cuda(), scale_b=torch.full((N,), 0.5).cuda())
    y = mt.linear(A.to(t).cuda(), B.to(t).cuda(), trans_b=True, out_dtype=torch.float32, **kw)
    assert torch.equal(y.double().cpu(), A.double() @ B.double().t())


@pytest.mark.parametrize("act", ACTS)
def test_no_contraction_gives_the_bias_alone(act):
    a = torch.empty(5, 0, dtype=torch.float16, device="cuda")
    b = torch.empty(0, 200, dtype=torch.float16, device="cuda")
    check(a, b, torch.linspace(-3, 3, 200).cuda(), act,
          torch.ones(5, 200, dtype=torch.float16, device="cuda"), preact=True)


def test_nothing_to_compute():
    a = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    b = torch.empty(64, 32, dtype=torch.float16, device="cuda")
    assert mt.linear(a, b).shape == (0, 32)
    assert mt.linear(b.t().contiguous()[:, :64], b[:, :0]).shape == (32, 0)


@pytest.mark.parametrize("M", [2, 50, 300])
def test_output_may_be_the_residual(M):
    g = torch.Generator().manual_seed(M)
    a, b = stored(g, M, 512, 512, torch.bfloat16), stored(g, 512, 640, 640, torch.bfloat16)
    res = stored(g, M, 640, 640, torch.bfloat16)
    want = mt.linear(a, b, residual=res, activation="gelu")
    got = mt.linear(a, b, residual=res, activation="gelu", out=res)
    assert got is res and torch.equal(got, want)


@pytest.mark.parametrize("M", [1, 33, 300])
def test_nan_infinity_and_zeros(M):
    """A NaN in a row of A reaches that row alone; so does an infinity."""
    g = torch.Generator().manual_seed(M)
    a = stored(g, M, 256, 256, torch.bfloat16)
    b = stored(g, 256, 384, 384, torch.bfloat16)
    clean = mt.linear(a, b, activation="silu")
    a[M // 2, 100] = float("nan")
    y = mt.linear(a, b, activation="silu")
    assert y[M // 2].isnan().all()
    a[M // 2, 100] = float("inf")
    z = mt.linear(a, b)
    assert not z[M // 2].isfinite().any()
    keep = [i for i in range(M) if i != M // 2]
    assert torch.equal(y[keep], clean[keep])
    assert (mt.linear(torch.zeros_like(a), b, activation="gelu_tanh") == 0).all()


def test_same_bits_every_time_on_any_stream_and_from_a_graph():
    g = torch.Generator().manual_seed(3)
    a, b = stored(g, 8, 4097, 4097, torch.float16), stored(g, 4097, 520, 520, torch.float16)
    want = mt.linear(a, b, activation="gelu")       # K split over a cluster, A copied
    torch.cuda.synchronize()
    for _ in range(5):
        assert torch.equal(mt.linear(a, b, activation="gelu"), want)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = mt.linear(a, b, activation="gelu")
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = mt.linear(a, b, activation="gelu")
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_a_wait_that_runs_out_is_reported():
    a = torch.ones(16, 2048, dtype=torch.bfloat16, device="cuda")
    b = torch.ones(2048, 256, dtype=torch.bfloat16, device="cuda")
    y = torch.full((16, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    p = mt.mt_linear_args(M=16, N=256, K=2048, A=a.data_ptr(), lda=2048, B=b.data_ptr(), ldb=256,
                          Y=y.data_ptr(), ldy=256, dtype=mt.MT_DTYPE_BF16,
                          out_dtype=mt.MT_DTYPE_BF16, fault_inject=1)
    torch.cuda.synchronize()
    assert mt.mt_linear(p, 0) == mt.MT_OK
    assert mt.mt_check_device_status(0) == mt.MT_ERR_TIMEOUT
    assert (y == 7).all()
    p.fault_inject = 0
    assert mt.mt_linear(p, 0) == mt.MT_OK
    assert mt.mt_check_device_status(0) == mt.MT_OK
    assert (y == 2048).all()


def test_a_wait_that_runs_out_on_cta_pairs_is_reported():
    """As above on the persistent kernel (90 tiles of 256 x 256)."""
    a = torch.ones(2304, 64, dtype=torch.bfloat16, device="cuda")
    b = torch.ones(64, 2560, dtype=torch.bfloat16, device="cuda")
    y = torch.full((2304, 2560), 7.0, dtype=torch.bfloat16, device="cuda")
    p = mt.mt_linear_args(M=2304, N=2560, K=64, A=a.data_ptr(), lda=64, B=b.data_ptr(), ldb=2560,
                          Y=y.data_ptr(), ldy=2560, dtype=mt.MT_DTYPE_BF16,
                          out_dtype=mt.MT_DTYPE_BF16, fault_inject=1)
    st, plan = mt.mt_linear_plan(p, 152)
    assert st == mt.MT_OK and plan.bm == 256
    torch.cuda.synchronize()
    assert mt.mt_linear(p, 0) == mt.MT_OK
    assert mt.mt_check_device_status(0) == mt.MT_ERR_TIMEOUT
    assert (y == 7).all()
    p.fault_inject = 0
    assert mt.mt_linear(p, 0) == mt.MT_OK
    assert mt.mt_check_device_status(0) == mt.MT_OK
    assert (y == 64).all()


def test_refusals():
    a = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(8, 16, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(bias=torch.zeros(16, device="cuda").bfloat16()),
               dict(residual=torch.zeros(4, 16, device="cuda")), dict(out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            mt.linear(a, b, **kw)
    with pytest.raises(TypeError):
        mt.linear(a.float(), b.float())
    with pytest.raises(TypeError):
        mt.linear(a, b.half())
    with pytest.raises(TypeError):
        mt.linear(a.cpu(), b)
    for kw in (dict(bias=torch.zeros(15, device="cuda")), dict(activation="tanh"),
               dict(trans_b=True), dict(scale_a=torch.ones(4, device="cuda"))):
        with pytest.raises(ValueError):
            mt.linear(a, b, **kw)
    q, w = a.to(E4M3), b.t().contiguous().to(E4M3)
    with pytest.raises(ValueError):
        mt.linear(q, w.t().contiguous().view(8, 16))
    with pytest.raises(TypeError):
        mt.linear(q, w, trans_b=True)
    with pytest.raises(mt.MtError) as e:
        mt.linear(a, b, out=torch.as_strided(a, (4, 16), (2, 1)))
    assert e.value.status == mt.MT_ERR_INVALID_ARG   # rows shorter than 16
