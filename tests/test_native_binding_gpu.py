"""GPU: the native marshalling as a Python extension: what a call does to
other threads and how it fails."""
import ctypes
import shutil
import subprocess
import threading
import time

import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from tiled_fp32_gemm_gb300 import layers

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def native():
    from tiled_fp32_gemm_gb300 import build
    build.build()
    x = torch.ones(2, 8, device="cuda", dtype=torch.bfloat16)
    mt.rms_norm(x, None)
    assert layers._native is not None


# An entry point that waits on the host, up to two seconds, for another thread.
HOLD = """
#include <time.h>
volatile int inside, go;
int hold(const void *args, void *stream) {
    (void)args; (void)stream;
    inside = 1;
    for (int i = 0; i < 2000; ++i) {
        struct timespec t = {0, 1000000};
        if (go) return 0;
        nanosleep(&t, 0);
    }
    return 8;
}
"""


@pytest.fixture
def held(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    (tmp_path / "hold.c").write_text(HOLD)
    subprocess.run([cc, "-shared", "-fPIC", "-o", str(tmp_path / "hold.so"),
                    str(tmp_path / "hold.c")], check=True)
    library = ctypes.CDLL(str(tmp_path / "hold.so"))
    address = ctypes.cast(library.hold, ctypes.c_void_p).value
    layers._native.use_library(address, address, address, address)
    yield library
    layers._point_native()


@pytest.mark.parametrize("call", ["rms_norm", "rms_norm_backward", "linear", "linear_backward"])
def test_other_threads_run_while_a_call_waits(held, call):
    """The call returns only because another Python thread got to run."""
    x = torch.ones(4, 8, device="cuda", dtype=torch.bfloat16)
    rstd = torch.ones(4, device="cuda")
    calls = {"rms_norm": lambda: mt.rms_norm(x, None, residual=x),
             "rms_norm_backward": lambda: mt.rms_norm_backward(x, x, None, rstd),
             "linear": lambda: mt.linear(x, x, trans_b=True),
             "linear_backward": lambda: mt.linear_backward(x, x, torch.ones_like(x).repeat(2, 1),
                                                           trans_b=True)}
    inside, go = (ctypes.c_int.in_dll(held, n) for n in ("inside", "go"))
    inside.value = go.value = 0

    def release():
        while not inside.value:
            time.sleep(0.001)
        go.value = 1

    other = threading.Thread(target=release)
    other.start()
    try:
        calls[call]()          # MtError (status 8) when nobody could release it
    finally:
        other.join()


def test_output_that_does_not_fit_raises_torchs_error(monkeypatch):
    """2^41 bytes of output from 32 MB of inputs: the allocation fails, with
    the exception it has everywhere else in torch, native or not."""
    a = torch.ones(1 << 20, 8, device="cuda", dtype=torch.bfloat16)
    for unload in (False, True):
        if unload:
            monkeypatch.setattr(layers, "_native", None)
        with pytest.raises(torch.OutOfMemoryError):
            mt.linear(a, a, trans_b=True)
