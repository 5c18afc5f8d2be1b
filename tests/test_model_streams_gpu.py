"""GPU: the residual joins and the vocabulary's loss on other streams, from two
streams at once, and captured into graphs that are replayed beside each other:
the same results as one call after the other."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    return mt.lib()


def operands(seed, T=300, d=264, V=9000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    draw = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    target = torch.randint(0, V, (T,), generator=g, device="cuda")
    return (draw(T, d), draw(T, d), draw(V, d) / 16, torch.rand(T, generator=g, device="cuda"),
            target, torch.tensor([seed], device="cuda"))


NAMES = ["layer_norm", "layer_norm_backward", "dropout", "linear_cross_entropy",
         "linear_cross_entropy_backward"]


def calls(stream, ops):
    x, r, vocab, f, target, seed = ops
    s = {} if stream is None else {"stream": stream}
    drop = dict(dropout=0.2, seed=seed, sequence=3)
    return {
        "layer_norm": lambda: mt.layer_norm(x, residual=r, **drop, **s),
        "layer_norm_backward": lambda: mt.layer_norm_backward(x, r, None, f, f, dh=r, **drop, **s),
        "dropout": lambda: (mt.dropout(x, 0.2, seed, residual=r, **s),),
        "linear_cross_entropy": lambda: mt.linear_cross_entropy(x, vocab, target, trans_b=True,
                                                                label_smoothing=0.1, **s),
        "linear_cross_entropy_backward": lambda: mt.linear_cross_entropy_backward(
            f, x, vocab, target, f + 9, trans_b=True, **s)}


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("where", ["another", "current", "default"])
def test_same_results_on_the_stream_given(name, where):
    ops = operands(1)
    want = calls(None, ops)[name]()
    torch.cuda.synchronize()
    other, outer = torch.cuda.Stream(), torch.cuda.Stream()
    if where == "current":
        got = calls(torch.cuda.current_stream().cuda_stream, ops)[name]()
    elif where == "default":
        with torch.cuda.stream(outer):
            got = calls(0, ops)[name]()
    else:
        got = calls(other.cuda_stream, ops)[name]()
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_two_streams_at_once(name):
    """Each call's scratch is its own."""
    sets = [operands(s) for s in (1, 2)]
    want = [calls(None, o)[name]() for o in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(calls(None, sets[i])[name]())
    torch.cuda.synchronize()
    for i, results in enumerate(got):
        assert all(same(r, want[i]) for r in results)


@pytest.mark.parametrize("name", NAMES)
def test_two_graphs_replayed_beside_each_other(name):
    """Two captured graphs of the same call on other operands, replayed in turn
    and from two streams at once, give what eager calls give."""
    sets = [operands(s) for s in (1, 2)]
    fresh = [operands(s) for s in (3, 4)]
    for o in sets:
        calls(None, o)[name]()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for o in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(calls(None, o)[name]())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in sets]
    for source in (sets, fresh):
        want = [calls(None, o)[name]() for o in source]
        for o, s in zip(sets, source):
            for a, b in zip(o, s):
                a.copy_(b)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs * 3, streams * 3):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(same(o, w) for o, w in zip(outs, want))


def test_results_do_not_depend_on_what_scratch_held():
    """Scratch is pool memory that other calls have used: filled with NaN before
    the call, the results are the same."""
    ops = operands(5)
    want = {n: calls(None, ops)[n]() for n in NAMES}
    big = operands(6, T=1024, V=40000)
    nan = torch.full((1024,), float("nan"), device="cuda")
    for name in NAMES:
        x, _, vocab, _, target, _ = big
        mt.linear_cross_entropy_backward(nan, x, vocab, target, nan, trans_b=True)
        mt.layer_norm_backward(x * float("nan"), x, None, nan, nan)
        assert same(calls(None, ops)[name](), want[name])
