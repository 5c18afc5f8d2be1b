"""GPU: the `stream` argument of the feed-forward calls: the same results as
on the current stream, in memory that no stream's pending work still uses.
Which block an output gets is the allocator's decision at the call, so it is
read off the addresses: nothing races here."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu

CYCLES = 100_000_000     # some 50 ms of the current stream


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


def operands():
    g = torch.Generator(device="cuda").manual_seed(4)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    return draw(256, 1024), draw(256, 1024), draw(512, 1024), torch.rand(256, generator=g, device="cuda")


def calls(stream):
    x, r, w, rstd = operands()
    bias, z = torch.ones(512, device="cuda"), x[:, :512].contiguous()
    s = {} if stream is None else {"stream": stream}
    return {
        "rms_norm": lambda: mt.rms_norm(x, None, residual=r, **s),
        "rms_norm e4m3": lambda: mt.rms_norm(x, None, out_dtype=torch.float8_e4m3fn, **s),
        "rms_norm_backward": lambda: mt.rms_norm_backward(x, r, None, rstd, dh=r, **s),
        "linear": lambda: mt.linear(x, w, bias=bias, activation="gelu", residual=z, trans_b=True,
                                    preact=True, **s),
        "linear_backward": lambda: mt.linear_backward(z, x, w, z=z, activation="silu",
                                                      trans_b=True, **s)}


NAMES = ["rms_norm", "rms_norm e4m3", "rms_norm_backward", "linear", "linear_backward"]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("where", ["another", "current", "default"])
def test_same_results_on_the_stream_given(name, where):
    want = calls(None)[name]()
    torch.cuda.synchronize()
    other, outer = torch.cuda.Stream(), torch.cuda.Stream()
    if where == "current":
        got = calls(torch.cuda.current_stream().cuda_stream)[name]()
    elif where == "default":
        call = calls(0)[name]
        with torch.cuda.stream(outer):
            torch.cuda.synchronize()
            got = call()
    else:
        call = calls(other.cuda_stream)[name]
        torch.cuda.synchronize()
        before = torch.cuda.current_stream()
        got = call()
        assert torch.cuda.current_stream() == before
        other.synchronize()
    torch.cuda.synchronize()
    assert same(want, got)


def test_given_outputs_are_used_and_work_is_on_the_stream():
    x, r, w, _ = operands()
    y = torch.zeros(256, 512, device="cuda", dtype=torch.bfloat16)
    want = mt.linear(x, w, trans_b=True)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(CYCLES)
    done = torch.cuda.Event()
    assert mt.linear(x, w, trans_b=True, out=y, stream=s.cuda_stream) is y
    with torch.cuda.stream(s):
        done.record()
    assert not done.query()                  # behind that stream's work, not this one's
    torch.cuda.current_stream().synchronize()
    assert not done.query()
    s.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("call", ["mt.linear", "mt.rms_norm"])
def test_outputs_are_not_put_where_the_current_stream_still_reads(call):
    """A block the current stream has given back, its last use still queued."""
    x, r, w, _ = operands()
    s = torch.cuda.Stream()
    f = {"mt.linear": lambda: mt.linear(x, r, trans_b=True, stream=s.cuda_stream),
         "mt.rms_norm": lambda: mt.rms_norm(x, None, stream=s.cuda_stream)[0]}[call]
    shape = (256, 256) if call == "mt.linear" else (256, 1024)
    f()                                      # whatever the call loads or allocates once
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.full(shape, 3.0, device="cuda", dtype=torch.bfloat16)
    seen = torch.empty_like(old)
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    seen.copy_(old)
    where = old.data_ptr()
    del old
    y = f()
    assert y.data_ptr() != where
    torch.cuda.synchronize()
    assert (seen == 3).all()


def test_outputs_are_kept_until_the_current_stream_has_read_them():
    x, r, w, _ = operands()
    s = torch.cuda.Stream()
    y = mt.linear(x, w, trans_b=True, stream=s.cuda_stream)
    s.synchronize()
    seen, where = torch.empty_like(y), y.data_ptr()
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    seen.copy_(y)
    del y
    z = mt.linear(x, w, trans_b=True, stream=s.cuda_stream)
    assert z.data_ptr() != where
    torch.cuda.synchronize()
    assert torch.equal(seen, z)


def test_refusals_are_the_same_on_another_stream():
    x, r, w, _ = operands()
    s = torch.cuda.Stream().cuda_stream
    with pytest.raises(TypeError):
        mt.rms_norm(x.cpu(), None, stream=s)
    with pytest.raises(ValueError):
        mt.linear(x, w, stream=s)
    with pytest.raises(mt.MtError) as e:
        mt.rms_norm(x, None, eps=-1.0, stream=s)
    assert e.value.status == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("call", ["sgemm", "gemm", "gemm_mixed"])
def test_products_take_their_output_from_the_stream_given(call):
    """The older calls, the same way."""
    x, r, _, _ = operands()
    a, b = x.float(), r.float().t().contiguous()
    bias = torch.ones(256, device="cuda")
    f = {"sgemm": lambda **k: mt.sgemm(a, b, **k),
         "gemm": lambda **k: mt.gemm(a, b, alpha=2.0, bias=bias, **k),
         "gemm_mixed": lambda **k: mt.gemm_mixed(x, r, trans_b=True, **k)}[call]
    s = torch.cuda.Stream()
    want = f()
    f(stream=s.cuda_stream)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    old = torch.full((256, 256), 3.0, device="cuda")
    seen = torch.empty_like(old)
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    seen.copy_(old)
    where = old.data_ptr()
    del old
    y = f(stream=s.cuda_stream)
    assert y.data_ptr() != where
    torch.cuda.synchronize()
    assert (seen == 3).all() and torch.equal(y, want)


def test_products_into_a_given_output_run_on_the_stream_given():
    """Nothing to allocate: straight to the stream, as always."""
    x, r, _, _ = operands()
    a, b = x.float(), r.float().t().contiguous()
    c = torch.zeros(256, 256, device="cuda")
    calls = [lambda s: mt.sgemm(a, b, out=c, stream=s), lambda s: mt.gemm(a, b, c, stream=s),
             lambda s: mt.gemm_mixed(x, r, c, trans_b=True, stream=s)]
    for f in calls:
        want = f(None).clone()
        c.zero_()
        s, done = torch.cuda.Stream(), torch.cuda.Event()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(CYCLES)
        assert f(s.cuda_stream) is c
        done.record(s)
        torch.cuda.current_stream().synchronize()
        assert not done.query()
        s.synchronize()
        assert torch.equal(c, want)
