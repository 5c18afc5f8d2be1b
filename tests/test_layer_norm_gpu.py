"""GPU: mt_layer_norm and mt_dropout against their definitions in 64 bits.

Tolerances (u = 2^-24 of fp32, s = 2^-11, 2^-8 or u of the storage type).  A
dropped-out value is one product with a rounded factor: e_x = 2 u |x / (1 - p)|;
with the residual's addition h is within e_h = e_x + u |h|, and s |h| more when
stored (fp16: half its subnormal step, 2^-25, at least).  Sums of a row are at
most 16 deep in a thread (d / 512 in the wide kernel) and 12 over threads and
warps, so the mean is within E = (32 + d / 512) u mean|h| + mean e_h, and with c =
|h - m| the variance within mean(2 c (E + e_h + 2 u c)) + (E + max e_h)^2 + (40 +
d / 512) u variance.  r is good to 4 u more, y to c r |w| (dr / r + 3 u) + (E +
e_h) r |w| + 2 u (|c r w| + |b|) before its rounding.
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


def rows_of(g, rows, d, pitch, dt, scale=1.0, offset=0.0):
    """rows x d values in a rows x pitch buffer whose other columns are NaN."""
    buf = torch.full((rows, pitch), float("nan"), dtype=dt)
    buf[:, :d] = (torch.randn(rows, d, generator=g) * scale + offset).to(dt)
    return buf.cuda()[:, :d]


def seed_of(value):
    return torch.tensor([value], dtype=torch.int64, device="cuda")


def philox(counter, key):
    """Philox4x32-10 on Python integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


@pytest.mark.parametrize("counter,key,want", [
    # The known answers published with the generator.
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))])
def test_reference_generator_gives_the_published_words(counter, key, want):
    assert tuple(philox(counter, key)) == want


def mask_of(rows, d, p, seed, sequence):
    """Which elements are kept, an element at a time in Python integers."""
    border = int(p * 2 ** 32)
    key = (seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF)
    words = [[w for b in range((d + 3) // 4)
              for w in philox((b, i, sequence & 0xFFFFFFFF, sequence >> 32), key)][:d]
             for i in range(rows)]
    return torch.tensor([[w >= border for w in r] for r in words], device="cuda").view(rows, d)


def mask_by_columns(rows, d, p, seed, sequence):
    """The same mask for larger sizes, in 64-bit integer tensors."""
    i64 = lambda v: torch.tensor(v, dtype=torch.int64, device="cuda")  # noqa: E731
    m32 = 0xFFFFFFFF
    at = torch.arange(rows * ((d + 3) // 4), device="cuda")
    blocks = (d + 3) // 4
    c = [at % blocks, at // blocks, i64(sequence & m32).expand_as(at),
         i64(sequence >> 32).expand_as(at)]
    k = [seed & m32, seed >> 32 & m32]
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(p1 >> 32 & m32) ^ c[1] ^ k[0], p1 & m32, (p0 >> 32 & m32) ^ c[3] ^ k[1], p0 & m32]
        k = [(k[0] + 0x9E3779B9) & m32, (k[1] + 0xBB67AE85) & m32]
    words = torch.stack(c, 1).view(rows, 4 * blocks)[:, :d]
    return words >= int(p * 2 ** 32)


def within(got, want, bound):
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} off, max excess " \
        f"{((got - want).abs() - bound).max().item():.3g}"


def stored_step(v, dt):
    least = 2.0 ** -25 if dt == torch.float16 else 0.0
    return (STEP[dt] * v.abs()).clamp(min=least)


def joined(x, res, keep, p):
    """(h, its bound before storage)."""
    v = torch.where(keep, x.double() / (1 - p), 0.0) if p else x.double()
    e = 2 * U * v.abs() if p else torch.zeros_like(v)
    if res is None:
        return v, e
    h = v + res.double()
    return h, e + U * h.abs()


def check(x, res, w, b, eps=1e-5, p=0.0, seed=0, sequence=0, **kw):
    rows, d = x.shape
    dt = x.dtype
    x0, res0 = x.clone(), None if res is None else res.clone()
    got = mt.layer_norm(x, w, b, residual=res, eps=eps, dropout=p, seed=seed_of(seed),
                        sequence=sequence, **kw)
    y, h, mean, rstd = got
    keep = mask_by_columns(rows, d, p, seed, sequence) if p else None
    H, eh = joined(x0, res0, keep, p)
    if res is not None or p:
        within(h, H, eh + stored_step(H, dt))
    else:
        assert h is x
    M = H.mean(1, keepdim=True) if d else H.new_zeros(rows, 1)
    E = (32 + d / 512) * U * H.abs().mean(1, keepdim=True) + eh.mean(1, keepdim=True)
    within(mean[:, None], M, E + U * M.abs())
    C = (H - M).abs()
    var = (C * C).mean(1, keepdim=True)
    dvar = (2 * C * (E + eh + 2 * U * C)).mean(1, keepdim=True) + \
        (E + eh.amax(1, keepdim=True)) ** 2 + (40 + d / 512) * U * var
    R = (var + eps) ** -0.5
    rel = 0.5 * dvar / (var + eps) * (1 + dvar / (var + eps)) + 4 * U
    within(rstd[:, None], R, 2 * rel * R)
    W = w.double() if w is not None else H.new_ones(d)
    B = b.double() if b is not None else H.new_zeros(d)
    Y = (H - M) * R * W + B
    bound = C * R * W.abs() * (2 * rel + 5 * U) + (E + eh) * R * W.abs() * (1 + 2 * rel) + \
        2 * U * B.abs()
    within(y, Y, bound + stored_step(Y, dt) + STEP[dt] * bound)
    return got


SIZES = [(1, 1), (1, 2), (2, 7), (3, 8), (5, 31), (4, 33), (7, 255), (9, 256), (3, 257), (2, 1000),
         (6, 1024), (5, 1025), (3, 3001), (2, 4096), (3, 8192), (2, 8200), (2, 16384), (2, 16400),
         (1, 20001), (153, 520)]


@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,d", SIZES)
def test_sizes(rows, d, dtype, p):
    g = torch.Generator().manual_seed(rows * 100003 + d)
    dt = DTYPES[dtype]
    for pad, other in ((0, False), (5, True)):
        x, r = rows_of(g, rows, d, d + pad, dt), rows_of(g, rows, d, d + pad, dt, 2.0)
        w = (1 + 0.1 * torch.randn(d, generator=g)).cuda().to(torch.float32 if other else dt)
        b = (0.1 * torch.randn(d, generator=g)).cuda().to(w.dtype)
        check(x, r, w, b, p=p, seed=7 + d, sequence=3)
        check(x, None, None if other else w, b if other else None, p=p, seed=-1 - d,
              sequence=2 ** 40 + 1)


@pytest.mark.parametrize("offset", [3.0, 1000.0])
@pytest.mark.parametrize("d", [64, 1000, 4096, 20000])
def test_a_common_offset_leaves_the_variance_its_digits(offset, d):
    g = torch.Generator().manual_seed(d)
    x = rows_of(g, 3, d, d, torch.float32, 1.0, offset)
    check(x, None, None, None)


@pytest.mark.parametrize("eps", [0.0, 1e-5])
def test_constant_rows(eps):
    """A variance of 0: r is 1 / sqrt(eps), or 0 without an eps, and y the bias."""
    x = torch.full((3, 520), 2.0, device="cuda").bfloat16()
    x[1] = 0.0
    b = torch.arange(520, device="cuda").float()
    y, _, mean, rstd = mt.layer_norm(x, None, b, eps=eps)
    assert torch.equal(y, b.bfloat16().expand(3, -1))
    assert torch.equal(mean, x[:, 0].float())
    want = 0.0 if eps == 0.0 else eps ** -0.5
    assert ((rstd - want).abs() <= 4 * U * want).all()


@pytest.mark.parametrize("d", [40, 300, 17000])
def test_nan_and_infinite_rows_keep_to_themselves(d):
    x = torch.randn(4, d, device="cuda")
    x[1, d // 2] = float("nan")
    x[2, d - 1] = float("inf")
    y, _, mean, rstd = mt.layer_norm(x)
    assert y[1].isnan().all() and rstd[1].isnan() and mean[1].isnan()
    assert y[2].isnan().all() and rstd[2].isnan() and not mean[2].isfinite()
    keep = torch.tensor([0, 3], device="cuda")
    want = mt.layer_norm(x[keep].contiguous())
    assert torch.equal(y[keep], want[0]) and torch.equal(rstd[keep], want[3])


def test_no_rows_and_no_columns():
    y, h, mean, rstd = mt.layer_norm(torch.empty(0, 8, device="cuda"))
    assert y.shape == (0, 8) and mean.shape == (0,)
    y, h, mean, rstd = mt.layer_norm(torch.empty(3, 0, device="cuda"), eps=0.25)
    assert torch.equal(mean.cpu(), torch.zeros(3)) and torch.equal(rstd.cpu(), torch.full((3,), 2.0))


@pytest.mark.parametrize("d", [64, 250, 20000])
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_in_place(d, p):
    """h in place of the residual or of x, y in place of x."""
    g = torch.Generator().manual_seed(d)
    x, r = rows_of(g, 5, d, d, torch.bfloat16), rows_of(g, 5, d, d, torch.bfloat16)
    kw = dict(dropout=p, seed=seed_of(5), sequence=1)
    want = mt.layer_norm(x, residual=r, **kw)
    for h_is, y_is in (("r", None), ("x", None), ("r", "x")):
        a, b = x.clone(), r.clone()
        out = a if y_is else None
        got = mt.layer_norm(a, residual=b, h_out=b if h_is == "r" else a, out=out, **kw)
        for u, v in zip(got, want):
            assert torch.equal(u, v)


# --- dropout -------------------------------------------------------------------
@pytest.mark.parametrize("seed,sequence", [(0, 0), (-1, 2 ** 64 - 1), (2 ** 62 + 12345, 2 ** 33 + 7)])
@pytest.mark.parametrize("rows,d,pad", [(3, 16, 0), (2, 19, 0), (5, 33, 3), (2, 300, 0), (1, 264, 8)])
def test_dropped_elements_are_the_generators(rows, d, pad, seed, sequence):
    x = torch.ones(rows, d + pad, device="cuda")[:, :d]
    for p in (0.25, 0.5):
        y = mt.dropout(x, p, seed_of(seed), sequence=sequence)
        keep = mask_of(rows, d, p, seed % 2 ** 64, sequence)
        assert torch.equal(y != 0, keep)
        assert torch.equal(y[keep], torch.full_like(y[keep], 1 / (1 - p)))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,d,pad", [(1, 1, 0), (3, 5, 2), (2, 8, 0), (17, 64, 0), (5, 250, 0),
                                        (40, 256, 8), (3, 1024, 0), (7, 2047, 1), (4, 2056, 0),
                                        (2, 8192, 0), (3, 20001, 0), (2, 40000, 0), (1300, 72, 0)])
def test_dropout_sizes(rows, d, pad, dtype):
    g = torch.Generator().manual_seed(rows + d)
    dt = DTYPES[dtype]
    x, r = rows_of(g, rows, d, d + pad, dt), rows_of(g, rows, d, d + pad, dt)
    for p, res in ((0.1, None), (0.9, r), (0.0, r)):
        y = mt.dropout(x, p, seed_of(rows - d), sequence=rows, residual=res)
        keep = mask_by_columns(rows, d, p, rows - d, rows)
        want, e = joined(x, res, keep, p)
        within(y, want, e + stored_step(want, dt))
        if res is None:
            assert not y[~keep].any()
        for target in (x, r) if res is not None else (x,):
            a, b = x.clone(), r.clone()
            got = mt.dropout(a, p, seed_of(rows - d), sequence=rows,
                             residual=None if res is None else b,
                             out=a if target is x else b)
            assert torch.equal(got, y)


def test_dropped_nan_and_infinity_are_zeros():
    x = torch.full((4, 512), float("nan"), device="cuda")
    x[1] = float("inf")
    y = mt.dropout(x, 0.5, seed_of(3))
    keep = mask_by_columns(4, 512, 0.5, 3, 0)
    assert torch.equal(y == 0, ~keep)


def test_share_of_dropped_elements():
    """2^22 independent words: within six standard deviations."""
    for p in (0.1, 0.5):
        y = mt.dropout(torch.ones(1024, 4096, device="cuda"), p, seed_of(11))
        n = y.numel()
        assert abs((y == 0).sum().item() - p * n) < 6 * (n * p * (1 - p)) ** 0.5


def test_seed_is_read_when_the_kernel_runs():
    """A captured graph whose seed advances drops other elements each time."""
    x, seed = torch.ones(64, 512, device="cuda"), seed_of(100)
    mt.dropout(x, 0.5, seed)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        y = mt.dropout(x, 0.5, seed)
        n = mt.layer_norm(x, residual=y, dropout=0.5, seed=seed, sequence=9)
        seed.add_(1)
    for turn in range(3):
        graph.replay()
        torch.cuda.synchronize()
        want = mt.dropout(x, 0.5, seed_of(100 + turn))
        assert torch.equal(y, want)
        m = mt.layer_norm(x, residual=want, dropout=0.5, seed=seed_of(100 + turn), sequence=9)
        assert all(torch.equal(a, b) for a, b in zip(n, m))
    assert seed.item() == 103
