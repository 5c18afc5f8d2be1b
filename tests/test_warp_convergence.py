"""Warp-wide instructions of the feed-forward kernels (PTX `.aligned`: every
lane executes the same one together) follow a point where the warp has met.
After a lane-dependent branch nothing but a warp barrier promises that, so it
stands in the source; which lanes reconverge on their own shows in no result."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "tiled_fp32_gemm_gb300", "csrc")


def source(name):
    """A source file without its comments, blanks run together."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    text = re.sub(r"//[^\n]*|/\*.*?\*/", " ", text, flags=re.S)
    return re.sub(r"\s+", " ", text)


def test_drain_reads_its_sums_with_a_whole_warp():
    """Lanes at or past the last column skip the stores of a block of rows
    (and the residual's loads); the next block's sums come from tensor memory
    by a warp-wide load."""
    text = source("linear.cuh")
    calls = [m.start() for m in re.finditer(r"\bsums\(t, v\);", text)]
    assert calls
    for at in calls:
        assert text[:at].rstrip().endswith("__syncwarp();")


def test_cluster_barrier_meets_the_warp_first():
    """Its callers arrive from lane-dependent branches (a store for the last
    columns alone, a bounded spin)."""
    body = re.search(r"void cluster_sync\(\) \{(.*?)\}", source("tcgen05.cuh")).group(1)
    assert body.index("__syncwarp();") < body.index("barrier.cluster.arrive.release.aligned")


def test_named_barrier_meets_the_warp_first():
    """bar.sync is barrier.sync.aligned; lane 0 alone has just written the
    row's sum or arrived on the stage's barrier."""
    text = source("rms_norm_grad.cu")
    calls = [m.start() for m in re.finditer(r'asm volatile\("bar\.sync', text)]
    assert calls
    for at in calls:
        assert text[:at].rstrip().endswith("__syncwarp(); if (warps > 1)")


def test_products_read_their_accumulator_with_a_whole_warp():
    """Each chunk of the drain ends in stores that rows past the last (or
    columns past it) skip, and the next begins with a warp-wide load."""
    text = source("tcgen05.cuh")
    body = text[text.index("store_accumulator("):]
    loops = body.split("for (int ch = 0; ch < BN / 32; ++ch)")[1:]
    assert len(loops) == 2
    assert loops[0].lstrip().startswith("{ float v[32]; tmem_ld32(")
    assert loops[0].split("return;")[0].rstrip(" }").endswith("__syncwarp();")
    assert loops[1].lstrip().startswith("{ float v[32]; __syncwarp(); tmem_ld32(")
