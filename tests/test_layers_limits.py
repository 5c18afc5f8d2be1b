"""Host-side limits of the feed-forward operators: sizes whose index
arithmetic would not fit are refused before anything is launched (the
pointers here are never dereferenced)."""
import pytest

import tiled_fp32_gemm_gb300 as mt
from tiled_fp32_gemm_gb300 import build as mt_build

try:
    import torch
    HAS_GPU = torch.cuda.is_available()
except Exception:  # pragma: no cover
    HAS_GPU = False

LONGEST = 2 ** 31 - 512     # columns of a norm's row
APART = 1 << 40             # bytes between made-up operands


@pytest.fixture(scope="module", autouse=True)
def built_library():
    mt_build.build()
    return mt.lib()


def norm_of(d, **change):
    """One row of d fp32 values, every operand far from the others."""
    a = mt.mt_rms_norm_args(rows=1, d=d, x=APART, ldx=d, residual=2 * APART, ldr=d,
                            weight=3 * APART, h=4 * APART, ldh=d, y=5 * APART, ldy=d,
                            rstd=6 * APART, eps=1e-6, dtype=mt.MT_DTYPE_F32,
                            out_dtype=mt.MT_DTYPE_F32, weight_dtype=mt.MT_DTYPE_F32)
    for k, v in change.items():
        setattr(a, k, v)
    return a


def norm_grad_of(d):
    return mt.mt_rms_norm_backward_args(rows=1, d=d, dy=APART, lddy=d, h=2 * APART, ldh=d,
                                        weight=3 * APART, rstd=4 * APART, dh=5 * APART, lddh=d,
                                        dx=6 * APART, lddx=d, dweight=7 * APART,
                                        dtype=mt.MT_DTYPE_F32, weight_dtype=mt.MT_DTYPE_F32)


def answers(d):
    e4m3 = dict(out_dtype=mt.MT_DTYPE_E4M3, scale=8 * APART)
    return [mt.mt_rms_norm(norm_of(d)), mt.mt_rms_norm(norm_of(d, **e4m3)),
            mt.mt_rms_norm_backward(norm_grad_of(d))]


@pytest.mark.parametrize("d", [LONGEST + 1, 2 ** 31 - 32, 2 ** 31 - 31, 2 ** 31 - 1])
def test_norms_refuse_rows_whose_columns_pass_32_bits(d):
    """Columns advance by 512 and are rounded up to strips of 32 in 32 bits:
    both stay below 2^31 up to 2^31 - 512 columns."""
    assert answers(d) == [mt.MT_ERR_INVALID_ARG] * 3


@pytest.mark.skipif(HAS_GPU, reason="made-up addresses")
def test_the_longest_row_is_taken():
    assert LONGEST - 1 + 512 == 2 ** 31 - 1 and LONGEST + 31 < 2 ** 31
    assert answers(LONGEST) == [mt.MT_ERR_NO_DEVICE] * 3


def test_plans_for_few_sms_launch_something():
    """A pair of CTAs wants two SMs; with one the tiles go to single CTAs."""
    for sms in (1, 2, 3, 7):
        for M in (1, 129, 256, 4096):
            a = mt.mt_linear_args(M=M, N=4096, K=512, lda=512, ldb=4096, ldy=4096,
                                  dtype=mt.MT_DTYPE_BF16, out_dtype=mt.MT_DTYPE_BF16)
            st, p = mt.mt_linear_plan(a, sms)
            assert st == mt.MT_OK and p.grid >= 1
            tiles = -(-M // p.bm) * -(-4096 // p.bn)
            assert p.grid == (2 * min(tiles, sms // 2) if p.bn == 256 else tiles * p.split_k)
            assert p.bn == 128 or sms >= 2
