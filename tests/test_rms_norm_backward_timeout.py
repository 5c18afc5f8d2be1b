"""The bounded waits of the norm gradient's staged rows: a wait that nothing
ends runs out, the call's stream stays usable and the device status says so."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from tiled_fp32_gemm_gb300 import build as mt_build


@pytest.fixture(scope="module", autouse=True)
def library():
    mt_build.build()
    return mt.lib()


def arguments(**change):
    a = mt.mt_rms_norm_backward_args(rows=4, d=16, dy=0x10000, lddy=16, h=0x20000, ldh=16,
                                     rstd=0x40000, dx=0x60000, lddx=16, dtype=mt.MT_DTYPE_F16)
    for k, v in change.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change", [dict(fault_inject=-1), dict(fault_inject=2),
                                    dict(reserved=1)])
def test_refuses_other_values(change):
    assert mt.mt_rms_norm_backward(arguments(**change)) == mt.MT_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("rows,d", [(1, 64), (5, 2048), (700, 4096), (3, 12288), (2, 16384)])
@pytest.mark.parametrize("carried", [False, True])
def test_a_wait_that_runs_out_is_reported(rows, d, carried):
    dy = torch.ones(rows, d, dtype=torch.bfloat16, device="cuda")
    h, r = dy.clone(), torch.ones(rows, device="cuda")
    dx, dw = torch.empty_like(dy), torch.empty(d, device="cuda")
    a = mt.mt_rms_norm_backward_args(
        rows=rows, d=d, dy=dy.data_ptr(), lddy=d, h=h.data_ptr(), ldh=d, rstd=r.data_ptr(),
        dh=h.data_ptr() if carried else None, lddh=d, dx=dx.data_ptr(), lddx=d,
        dweight=dw.data_ptr(), dtype=mt.MT_DTYPE_BF16, fault_inject=1)
    torch.cuda.synchronize()
    assert mt.mt_check_device_status(0) == mt.MT_OK
    assert mt.mt_rms_norm_backward(a, 0) == mt.MT_OK
    assert mt.mt_check_device_status(0) == mt.MT_ERR_TIMEOUT
    a.fault_inject = 0
    assert mt.mt_rms_norm_backward(a, 0) == mt.MT_OK
    assert mt.mt_check_device_status(0) == mt.MT_OK
    # g - xhat * mean(g * xhat) is 0 for ones; dweight counts the rows.
    assert (dx == (1 if carried else 0)).all() and (dw == rows).all()


@pytest.mark.gpu
def test_rows_that_are_not_staged_wait_for_nothing():
    dy = torch.ones(4, 1001, dtype=torch.bfloat16, device="cuda")
    h, r, dx = dy.clone(), torch.ones(4, device="cuda"), torch.empty_like(dy)
    a = mt.mt_rms_norm_backward_args(
        rows=4, d=1001, dy=dy.data_ptr(), lddy=1001, h=h.data_ptr(), ldh=1001, rstd=r.data_ptr(),
        dx=dx.data_ptr(), lddx=1001, dtype=mt.MT_DTYPE_BF16, fault_inject=1)
    torch.cuda.synchronize()
    assert mt.mt_rms_norm_backward(a, 0) == mt.MT_OK
    assert mt.mt_check_device_status(0) == mt.MT_OK
