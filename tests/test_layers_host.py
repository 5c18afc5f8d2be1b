"""Host-side checks of the feed-forward operators' C entry points: argument
errors and aliasing are refused before anything is launched (the pointers
here are never dereferenced), and without a GPU a valid call reports that."""
import ctypes

import pytest

import tiled_fp32_gemm_gb300 as mt
from tiled_fp32_gemm_gb300 import build as mt_build

try:
    import torch
    HAS_GPU = torch.cuda.is_available()
except Exception:  # pragma: no cover
    HAS_GPU = False


@pytest.fixture(scope="module", autouse=True)
def built_library():
    mt_build.build()
    return mt.lib()


CLASSES = (mt.mt_rms_norm_args, mt.mt_rms_norm_backward_args, mt.mt_linear_args,
           mt.mt_linear_backward_args)


def norm_args(**change):
    a = mt.mt_rms_norm_args(rows=4, d=16, x=0x10000, ldx=16, residual=0x20000, ldr=16,
                            weight=0x30000, h=0x40000, ldh=16, y=0x50000, ldy=16, scale=None,
                            rstd=0x60000, eps=1e-6, dtype=mt.MT_DTYPE_BF16,
                            out_dtype=mt.MT_DTYPE_BF16, weight_dtype=mt.MT_DTYPE_F32)
    for k, v in change.items():
        setattr(a, k, v)
    return a


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(d=-1), dict(rows=1 << 31), dict(d=1 << 31), dict(x=None), dict(y=None),
    dict(ldx=15), dict(ldr=15), dict(ldh=15), dict(ldy=15), dict(dtype=0), dict(dtype=9),
    dict(dtype=mt.MT_DTYPE_E4M3), dict(out_dtype=mt.MT_DTYPE_F16), dict(out_dtype=0),
    dict(weight_dtype=mt.MT_DTYPE_F16), dict(eps=-1e-6), dict(eps=INF), dict(eps=NAN),
    dict(scale=0x70000), dict(out_dtype=mt.MT_DTYPE_E4M3), dict(x=0x10001), dict(weight=0x30002),
    dict(rstd=0x60002), dict(ldx=1 << 60), dict(out_dtype=mt.MT_DTYPE_E4M3, scale=0x70002)])
def test_norm_refuses_invalid_arguments(change):
    assert mt.mt_rms_norm(norm_args(**change)) == mt.MT_ERR_INVALID_ARG


def test_norm_refuses_no_arguments():
    assert mt.lib().mt_rms_norm(None, None) == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(h=0x10002), dict(h=0x20010), dict(h=0x20000, ldh=32), dict(y=0x20000), dict(y=0x40000),
    dict(y=0x10010), dict(h=0x30000), dict(y=0x30010), dict(rstd=0x50000), dict(rstd=0x10004),
    dict(out_dtype=mt.MT_DTYPE_E4M3, scale=0x60000),
    dict(out_dtype=mt.MT_DTYPE_E4M3, scale=0x70000, y=0x10000, ldy=16)])
def test_norm_refuses_overlap(change):
    assert mt.mt_rms_norm(norm_args(**change)) == mt.MT_ERR_ALIAS


@pytest.mark.skipif(HAS_GPU, reason="made-up addresses")
@pytest.mark.parametrize("change", [dict(), dict(h=0x20000), dict(h=0x10000), dict(y=0x10000),
                                    dict(residual=None, h=None, weight=None, rstd=None),
                                    dict(out_dtype=mt.MT_DTYPE_E4M3, scale=0x70000)])
def test_norm_without_a_device(change):
    assert mt.mt_rms_norm(norm_args(**change)) == mt.MT_ERR_NO_DEVICE


def test_norm_of_no_rows_is_nothing():
    assert mt.mt_rms_norm(norm_args(rows=0)) == mt.MT_OK


def norm_grad_args(**change):
    a = mt.mt_rms_norm_backward_args(rows=4, d=16, dy=0x10000, lddy=16, h=0x20000, ldh=16,
                                     weight=0x30000, rstd=0x40000, dh=0x50000, lddh=16,
                                     dx=0x60000, lddx=16, dweight=0x70000,
                                     dtype=mt.MT_DTYPE_F16, weight_dtype=mt.MT_DTYPE_F16)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(d=1 << 31), dict(dy=None), dict(h=None), dict(rstd=None), dict(dx=None),
    dict(lddy=15), dict(ldh=1), dict(lddh=0), dict(lddx=15), dict(dtype=mt.MT_DTYPE_E4M3),
    dict(weight_dtype=mt.MT_DTYPE_BF16), dict(dweight=0x70002), dict(dx=0x60001)])
def test_norm_backward_refuses_invalid_arguments(change):
    assert mt.mt_rms_norm_backward(norm_grad_args(**change)) == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(dx=0x10002), dict(dx=0x50000, lddx=32), dict(dx=0x20000), dict(dx=0x30000),
    dict(dx=0x40000), dict(dweight=0x60000), dict(dweight=0x10004), dict(dweight=0x20000),
    dict(dweight=0x30000), dict(dweight=0x40000), dict(dweight=0x50000)])
def test_norm_backward_refuses_overlap(change):
    assert mt.mt_rms_norm_backward(norm_grad_args(**change)) == mt.MT_ERR_ALIAS


@pytest.mark.skipif(HAS_GPU, reason="made-up addresses")
@pytest.mark.parametrize("change", [dict(), dict(dx=0x10000), dict(dx=0x50000), dict(dh=None),
                                    dict(weight=None, dweight=None), dict(rows=0)])
def test_norm_backward_without_a_device(change):
    assert mt.mt_rms_norm_backward(norm_grad_args(**change)) == mt.MT_ERR_NO_DEVICE


def linear_args(**change):
    a = mt.mt_linear_args(M=4, N=16, K=32, A=0x10000, lda=32, B=0x20000, ldb=16, Y=0x30000,
                          ldy=16, Z=0x40000, ldz=16, residual=0x50000, ldr=16, bias=0x60000,
                          dtype=mt.MT_DTYPE_BF16, out_dtype=mt.MT_DTYPE_BF16,
                          activation=mt.MT_ACT_SILU)
    for k, v in change.items():
        setattr(a, k, v)
    return a


E4M3 = dict(dtype=mt.MT_DTYPE_E4M3, trans_b=1, ldb=32, scale_a=0x70000, scale_b=0x80000)


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 31), dict(A=None), dict(B=None),
    dict(Y=None), dict(lda=31), dict(ldb=15), dict(trans_b=1), dict(trans_b=2), dict(ldy=15),
    dict(ldz=15), dict(ldr=15), dict(dtype=mt.MT_DTYPE_F32), dict(dtype=0),
    dict(out_dtype=mt.MT_DTYPE_F16), dict(out_dtype=mt.MT_DTYPE_E4M3), dict(activation=5),
    dict(activation=-1), dict(bias=0x60002), dict(A=0x10001), dict(Y=0x30001),
    dict(scale_a=0x70000), dict(reserved=1), dict(fault_inject=2),
    {**E4M3, "trans_b": 0}, {**E4M3, "scale_a": None}, {**E4M3, "scale_b": None},
    {**E4M3, "scale_b": 0x80002}, {**E4M3, "out_dtype": mt.MT_DTYPE_E4M3}])
def test_linear_refuses_invalid_arguments(change):
    assert mt.mt_linear(linear_args(**change)) == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(Y=0x10000), dict(Y=0x20010), dict(Y=0x50002), dict(Y=0x50000, ldy=32), dict(Y=0x40000),
    dict(Y=0x60000), dict(Z=0x50000), dict(Z=0x10000), dict(Z=0x20000), dict(Z=0x60000),
    {**E4M3, "Y": 0x70000}, {**E4M3, "Z": 0x80000}])
def test_linear_refuses_overlap(change):
    assert mt.mt_linear(linear_args(**change)) == mt.MT_ERR_ALIAS


@pytest.mark.skipif(HAS_GPU, reason="made-up addresses")
@pytest.mark.parametrize("change", [dict(), dict(Y=0x50000), dict(Z=None, residual=None, bias=None),
                                    dict(K=0, A=None, B=None), dict(trans_b=1, ldb=32),
                                    dict(out_dtype=mt.MT_DTYPE_F32), E4M3,
                                    {**E4M3, "A": 0x10001, "lda": 33}])
def test_linear_without_a_device(change):
    assert mt.mt_linear(linear_args(**change)) == mt.MT_ERR_NO_DEVICE


@pytest.mark.parametrize("change", [dict(M=0), dict(N=0)])
def test_linear_of_nothing(change):
    assert mt.mt_linear(linear_args(**change)) == mt.MT_OK


def linear_plan(M, N, K, sms=152, **change):
    trans = change.get("trans_b", 0)
    a = linear_args(M=M, N=N, K=K, lda=max(K, 1), ldb=max(K if trans else N, 1), ldy=N, ldz=N,
                    ldr=N)
    for k, v in change.items():
        setattr(a, k, v)
    st, p = mt.mt_linear_plan(a, sms)
    assert st == mt.MT_OK
    return p.as_dict()


def test_linear_plans_cover_the_product():
    """Whatever the sizes: the tiles cover Y, slices of K are no more than
    its K tiles and no more than a cluster holds, shared memory fits."""
    for M in (1, 15, 16, 17, 33, 64, 65, 128, 129, 500, 4096, 8192):
        for N in (1, 127, 128, 129, 4096, 11000):
            for K in (0, 1, 64, 65, 1000, 8192):
                for change in (dict(), dict(trans_b=1), E4M3):
                    p = linear_plan(M, N, K, **{**change, "ldb": max(N, K, 1)})
                    tiles = -(-M // p["bm"]) * -(-N // p["bn"])
                    if p["bn"] == 128:
                        assert p["grid"] == tiles * p["split_k"]
                    assert 1 <= p["split_k"] <= max(1, min(8, -(-K // p["bk"])))
                    assert p["smem_bytes"] <= 227 * 1024


def test_linear_plan_reports_copies():
    """Rows TMA cannot read in place are copied into rows of whole 128-byte
    lines: 16-byte bases and pitches are read in place."""
    assert linear_plan(64, 64, 64)["workspace_bytes"] == 0
    p = linear_plan(64, 64, 65, lda=65)      # A's rows are 130 bytes
    assert p["vec_ab"] == 0 and p["workspace_bytes"] == 64 * 256
    p = linear_plan(64, 64, 64, A=0x10002)
    assert p["vec_ab"] == 0 and p["workspace_bytes"] == 64 * 128
    p = linear_plan(64, 65, 64)              # B's rows are 130 bytes
    assert p["workspace_bytes"] == 64 * 256
    p = linear_plan(64, 64, 72, **{**E4M3, "lda": 72, "ldb": 72})
    assert p["workspace_bytes"] == 2 * 64 * 128


def linear_grad_args(**change):
    a = mt.mt_linear_backward_args(M=4, N=16, K=32, dY=0x10000, lddy=16, Z=0x20000, ldz=16,
                                   A=0x30000, lda=32, B=0x40000, ldb=16, dA=0x50000, ldda=32,
                                   dB=0x60000, lddb=16, dbias=0x70000, dtype=mt.MT_DTYPE_F16,
                                   db_dtype=mt.MT_DTYPE_F16, activation=mt.MT_ACT_GELU)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(N=1 << 31), dict(K=-1), dict(dY=None), dict(Z=None), dict(A=None),
    dict(B=None), dict(lddy=15), dict(ldz=15), dict(lda=31), dict(ldb=15), dict(ldda=31),
    dict(lddb=15), dict(trans_b=1), dict(trans_b=-1), dict(dtype=mt.MT_DTYPE_E4M3),
    dict(dtype=mt.MT_DTYPE_F32), dict(db_dtype=mt.MT_DTYPE_BF16), dict(activation=7),
    dict(dbias=0x70001), dict(dB=0x60002, db_dtype=mt.MT_DTYPE_F32)])
def test_linear_backward_refuses_invalid_arguments(change):
    assert mt.mt_linear_backward(linear_grad_args(**change)) == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(dA=0x10000), dict(dA=0x20000), dict(dA=0x30000), dict(dA=0x40000), dict(dA=0x60000),
    dict(dA=0x70000), dict(dB=0x10000), dict(dB=0x20000), dict(dB=0x30000), dict(dB=0x40000),
    dict(dB=0x70000), dict(dbias=0x10000), dict(dbias=0x20004)])
def test_linear_backward_refuses_overlap(change):
    assert mt.mt_linear_backward(linear_grad_args(**change)) == mt.MT_ERR_ALIAS


@pytest.mark.skipif(HAS_GPU, reason="made-up addresses")
@pytest.mark.parametrize("change", [
    dict(), dict(activation=0, Z=None), dict(dA=None, B=None), dict(dB=None, A=None),
    dict(dbias=None), dict(M=0), dict(trans_b=1, ldb=32, lddb=32),
    dict(db_dtype=mt.MT_DTYPE_F32)])
def test_linear_backward_without_a_device(change):
    assert mt.mt_linear_backward(linear_grad_args(**change)) == mt.MT_ERR_NO_DEVICE


def test_linear_backward_of_nothing():
    assert mt.mt_linear_backward(linear_grad_args(dA=None, dB=None, dbias=None)) == mt.MT_OK
    assert mt.mt_linear_backward(linear_grad_args(K=0, dbias=None)) == mt.MT_OK


def test_packed_arguments_match_the_structure():
    """The binding's one-call packing lays the fields out as the structure."""
    from tiled_fp32_gemm_gb300 import layers
    for cls in CLASSES:
        values = [i + 1 for i in range(len(cls._fields_))]
        a = cls.from_buffer_copy(layers._packer(cls)(*values))
        for (name, _), v in zip(cls._fields_, values):
            assert getattr(a, name) == v, name


def test_arguments_have_the_c_layout(tmp_path):
    """sizeof and every field offset agree with the C header."""
    import os
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    cuda = os.path.join(os.path.dirname(os.path.dirname(mt_build.nvcc())), "include")
    lines, want = [], []
    for cls in CLASSES:
        n = cls.__name__
        lines.append(f'printf("%zu\\n", sizeof({n}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({n}, {f}));')
            want.append(getattr(cls, f).offset)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "mt_layers.h"\n'
                   'int main(void) {' + "\n".join(lines) + 'return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    "-I", cuda, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert [int(v) for v in out.split()] == want


def test_linear_plans_hold_their_tile_indices_in_32_bits():
    """256 x 256 tiles go to CTA pairs up to 2^28 - 1 of them; past that to the
    128 x 128 tiles of the split kernel, whose grid is refused past 2^31 - 1."""
    def status(M, N):
        a = linear_args(M=M, N=N, K=64, lda=64, ldb=N, ldy=N, ldz=N, ldr=N)
        return mt.mt_linear_plan(a, 152)
    st, p = status(2 ** 22 - 256, 2 ** 22)             # 2^28 - 2^14 pair tiles
    assert st == mt.MT_OK and p.bn == 256
    st, p = status(2 ** 22, 2 ** 22)                   # 2^28
    assert st == mt.MT_OK and p.bn == 128 and p.grid == 2 ** 30
    st, _ = status(2 ** 23, 2 ** 22)                   # a grid of 2^31
    assert st == mt.MT_ERR_UNSUPPORTED
