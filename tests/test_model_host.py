"""Host-side checks of the residual joins' and the vocabulary loss's C entry
points (include/mt_model.h): argument errors and aliasing are refused before
anything is launched (the pointers here are never dereferenced), and without a
GPU a valid call reports that; the binding's argument structures have the C
layout, and its own refusals say what is wrong."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from tiled_fp32_gemm_gb300 import build as mt_build, layers, model

HAS_GPU = torch.cuda.is_available()
INF, NAN = float("inf"), float("nan")
BF16, F16, F32 = 2, 1, mt.MT_DTYPE_F32

CLASSES = (mt.mt_layer_norm_args, mt.mt_layer_norm_backward_args, mt.mt_dropout_args,
           mt.mt_linear_cross_entropy_args, mt.mt_linear_cross_entropy_backward_args)


@pytest.fixture(scope="module", autouse=True)
def built_library():
    mt_build.build()
    return mt.lib()


def norm(**change):
    a = dict(rows=4, d=16, x=0x10000, ldx=16, residual=0x20000, ldr=16, weight=0x30000,
             bias=0x31000, h=0x40000, ldh=16, y=0x50000, ldy=16, mean=0x60000, rstd=0x61000,
             seed=0x70000, sequence=1, dropout=0.1, eps=1e-5, dtype=BF16, weight_dtype=F32)
    return mt.mt_layer_norm(mt.mt_layer_norm_args(**{**a, **change}))


def norm_grad(**change):
    a = dict(rows=4, d=16, dy=0x10000, lddy=16, h=0x20000, ldh=16, weight=0x30000, mean=0x31000,
             rstd=0x32000, dh=0x40000, lddh=16, dx=0x50000, lddx=16, dresidual=0x60000, lddres=16,
             dweight=0x70000, dbias=0x71000, seed=0x80000, sequence=1, dropout=0.1, dtype=BF16,
             weight_dtype=F32)
    return mt.mt_layer_norm_backward(mt.mt_layer_norm_backward_args(**{**a, **change}))


def drop(**change):
    a = dict(rows=4, d=16, x=0x10000, ldx=16, residual=0x20000, ldr=16, y=0x30000, ldy=16,
             seed=0x40000, sequence=1, p=0.1, dtype=BF16)
    return mt.mt_dropout(mt.mt_dropout_args(**{**a, **change}))


def loss(**change):
    a = dict(T=4, K=16, V=32, A=0x10000, lda=16, B=0x20000, ldb=32, target=0x30000, loss=0x40000,
             lse=0x41000, ignore_index=-100, label_smoothing=0.1, z_loss=1e-4, trans_b=0,
             dtype=BF16)
    return mt.mt_linear_cross_entropy(mt.mt_linear_cross_entropy_args(**{**a, **change}))


def loss_grad(**change):
    a = dict(T=4, K=16, V=32, dloss=0x90000, A=0x10000, lda=16, B=0x20000, ldb=32, target=0x30000,
             lse=0x41000, dA=0x50000, ldda=16, dB=0x60000, lddb=32, ignore_index=-100,
             label_smoothing=0.1, z_loss=1e-4, trans_b=0, dtype=BF16, db_dtype=F32)
    return mt.mt_linear_cross_entropy_backward(
        mt.mt_linear_cross_entropy_backward_args(**{**a, **change}))


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(d=-1), dict(rows=1 << 31), dict(d=(1 << 31) - 4095), dict(x=None),
    dict(y=None), dict(ldx=15), dict(ldr=15), dict(ldh=15), dict(ldy=15), dict(dtype=0),
    dict(dtype=mt.MT_DTYPE_E4M3), dict(weight_dtype=F16), dict(weight=None, weight_dtype=F16),
    dict(eps=-1e-6), dict(eps=INF), dict(eps=NAN), dict(dropout=1.0), dict(dropout=-0.1),
    dict(dropout=NAN), dict(seed=None), dict(seed=0x70004), dict(x=0x10001), dict(bias=0x31002),
    dict(rstd=0x61002), dict(ldx=1 << 60), dict(reserved=1)])
def test_norm_refuses(change):
    assert norm(**change) == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(h=0x10002), dict(h=0x20010), dict(h=0x20000, ldh=32), dict(y=0x20000), dict(y=0x40000),
    dict(y=0x10010), dict(h=0x30000), dict(y=0x31010), dict(rstd=0x50000), dict(mean=0x61000),
    dict(mean=0x10004), dict(y=0x70000), dict(rstd=0x70004)])
def test_norm_refuses_overlap(change):
    assert norm(**change) == mt.MT_ERR_ALIAS


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(d=(1 << 31) - 4095), dict(dy=None), dict(h=None), dict(dx=None),
    dict(mean=None), dict(rstd=None), dict(lddy=15), dict(lddh=15), dict(lddres=15),
    dict(dtype=9), dict(weight_dtype=F16), dict(dropout=1.0), dict(dropout=0.0), dict(seed=None),
    dict(fault_inject=2), dict(fault_inject=-1), dict(reserved=1), dict(dbias=0x71002)])
def test_norm_gradient_refuses(change):
    assert norm_grad(**change) == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    dict(dx=0x20000), dict(dx=0x10010), dict(dresidual=0x20000), dict(dresidual=0x50000),
    dict(dx=0x40000, lddx=32), dict(dweight=0x71000), dict(dweight=0x50000), dict(dbias=0x60000),
    dict(dbias=0x30000), dict(dweight=0x10000), dict(dx=0x80000), dict(dresidual=0x31000)])
def test_norm_gradient_refuses_overlap(change):
    assert norm_grad(**change) == mt.MT_ERR_ALIAS


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(d=-1), dict(d=(1 << 31) - 4095), dict(x=None), dict(y=None), dict(ldr=15),
    dict(dtype=mt.MT_DTYPE_E4M3), dict(p=1.0), dict(p=-1e-9), dict(p=NAN), dict(seed=None),
    dict(reserved=1), dict(y=0x30001)])
def test_dropout_refuses(change):
    assert drop(**change) == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(y=0x10002), dict(y=0x20000, ldy=32), dict(y=0x40000)])
def test_dropout_refuses_overlap(change):
    assert drop(**change) == mt.MT_ERR_ALIAS


@pytest.mark.parametrize("change", [
    dict(T=-1), dict(K=-1), dict(V=-1), dict(V=0), dict(T=1 << 31), dict(V=1 << 31), dict(A=None),
    dict(B=None), dict(target=None), dict(lse=None), dict(lda=15), dict(ldb=31),
    dict(trans_b=1, ldb=15), dict(trans_b=2), dict(dtype=F32), dict(dtype=mt.MT_DTYPE_E4M3),
    dict(label_smoothing=-0.1), dict(label_smoothing=1.1), dict(label_smoothing=NAN),
    dict(z_loss=-1.0), dict(z_loss=INF), dict(z_loss=NAN), dict(reserved=1),
    dict(target=0x30004)])
def test_loss_refuses(change):
    assert loss_grad(**change) == mt.MT_ERR_INVALID_ARG
    assert loss(**change) == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(dloss=None), dict(db_dtype=F16), dict(ldda=15),
                                    dict(lddb=31), dict(dA=0x50001)])
def test_loss_gradient_refuses(change):
    assert loss_grad(**change) == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(fault_inject=2), dict(loss=None), dict(loss=0x40002)])
def test_loss_alone_refuses(change):
    assert loss(**change) == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(loss=0x41000), dict(lse=0x10010), dict(loss=0x20000),
                                    dict(lse=0x30010)])
def test_loss_refuses_overlap(change):
    assert loss(**change) == mt.MT_ERR_ALIAS


@pytest.mark.parametrize("change", [
    dict(dA=0x10000), dict(dB=0x20000), dict(dA=0x60010), dict(dB=0x41000), dict(dA=0x90000),
    dict(dB=0x30000)])
def test_loss_gradient_refuses_overlap(change):
    assert loss_grad(**change) == mt.MT_ERR_ALIAS


def test_no_arguments():
    for name in model.SIGNATURES:
        assert getattr(mt.lib(), name)(None, None) == mt.MT_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [
    lambda: norm(rows=0), lambda: norm_grad(d=0), lambda: norm_grad(rows=0, dweight=None, dbias=None),
    lambda: drop(rows=0), lambda: drop(d=0, seed=None), lambda: loss(T=0), lambda: loss(T=0, V=0),
    lambda: loss_grad(T=0, dB=None), lambda: loss_grad(K=0), lambda: loss_grad(dA=None, dB=None)])
def test_nothing_to_do(call):
    assert call() == mt.MT_OK


@pytest.mark.skipif(HAS_GPU, reason="made-up addresses")
@pytest.mark.parametrize("call", [
    norm, lambda: norm(h=0x20000), lambda: norm(h=0x10000), lambda: norm(y=0x10000),
    lambda: norm(residual=None, h=None, weight=None, bias=None, mean=None, rstd=None, seed=None,
                 dropout=0.0), norm_grad, lambda: norm_grad(dx=0x10000, dresidual=0x40000),
    lambda: norm_grad(dresidual=None), lambda: norm_grad(dropout=0.0, dresidual=None, seed=None),
    drop, lambda: drop(y=0x10000), lambda: drop(y=0x20000), lambda: drop(p=0.0), loss,
    lambda: loss(trans_b=1), loss_grad, lambda: loss_grad(dA=None), lambda: loss_grad(T=0)])
def test_without_a_device(call):
    assert call() == mt.MT_ERR_NO_DEVICE


def test_packed_arguments_are_the_structures_fields():
    for cls in CLASSES:
        values = [i + 1 for i in range(len(cls._fields_))]
        a = cls.from_buffer_copy(layers._packer(cls)(*values))
        for (name, _), v in zip(cls._fields_, values):
            assert getattr(a, name) == v, name


def test_arguments_have_the_c_layout(tmp_path):
    """sizeof and every field offset agree with the C header."""
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
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "mt_model.h"\n'
                   'int main(void) {' + "\n".join(lines) + 'return 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run([cc, "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"),
                    "-I", cuda, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert [int(v) for v in out.split()] == want


def test_torch_calls_refuse_cpu_tensors():
    x, v = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: mt.layer_norm(x), lambda: mt.dropout(x, 0.1, v[:1]),
                 lambda: mt.layer_norm_backward(x, x, None, x[:, 0], x[:, 0]),
                 lambda: mt.linear_cross_entropy(x.half(), x.half(), v),
                 lambda: mt.linear_cross_entropy_backward(x[:, 0], x.half(), x.half(), v, x[:, 0])):
        with pytest.raises(TypeError):
            call()


@pytest.mark.gpu
def test_torch_calls_refuse():
    x = torch.zeros(4, 16, device="cuda", dtype=torch.bfloat16)
    f, seed = torch.zeros(16, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    t, s = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    b = torch.zeros(32, 16, device="cuda", dtype=torch.bfloat16)
    for error, call in [
            (TypeError, lambda: mt.layer_norm(x, f, x[0])),            # weight and bias types
            (TypeError, lambda: mt.layer_norm(x.double())),
            (ValueError, lambda: mt.layer_norm(x, f[:8])),
            (ValueError, lambda: mt.layer_norm(x, residual=x[:2])),
            (ValueError, lambda: mt.layer_norm(x, h_out=x)),
            (TypeError, lambda: mt.layer_norm(x, dropout=0.1)),
            (TypeError, lambda: mt.layer_norm(x, dropout=0.1, seed=3)),
            (TypeError, lambda: mt.layer_norm(x, dropout=0.1, seed=t)),
            (ValueError, lambda: mt.layer_norm(x, dropout=1.0, seed=seed)),
            (ValueError, lambda: mt.dropout(x, 0.1, seed, sequence=-1)),
            (ValueError, lambda: mt.dropout(x, 0.1, seed, sequence=2 ** 64)),
            (ValueError, lambda: mt.dropout(x, float("nan"), seed)),
            (TypeError, lambda: mt.dropout(x, 0.1, None)),
            (ValueError, lambda: mt.dropout(x.t(), 0.1, seed)),
            (ValueError, lambda: mt.layer_norm_backward(x, x, None, s[:2], s)),
            (mt.MtError, lambda: mt.dropout(x, 0.1, seed, out=torch.as_strided(x, (4, 16), (8, 1)))),
            (TypeError, lambda: mt.linear_cross_entropy(x, b, t.int(), trans_b=True)),
            (ValueError, lambda: mt.linear_cross_entropy(x, b, t[:3], trans_b=True)),
            (ValueError, lambda: mt.linear_cross_entropy(x, b, t)),
            (ValueError, lambda: mt.linear_cross_entropy(x, b[:0], t, trans_b=True)),
            (ValueError, lambda: mt.linear_cross_entropy(x, b, t, trans_b=True, label_smoothing=2)),
            (ValueError, lambda: mt.linear_cross_entropy(x, b, t, trans_b=True, z_loss=-1)),
            (TypeError, lambda: mt.linear_cross_entropy(x.float(), b, t, trans_b=True)),
            (TypeError, lambda: mt.linear_cross_entropy_backward(s, x, b, t, s, trans_b=True,
                                                                 db_dtype=torch.float16)),
            (TypeError, lambda: mt.linear_cross_entropy_backward(s.half(), x, b, t, s,
                                                                 trans_b=True))]:
        with pytest.raises(error):
            call()
