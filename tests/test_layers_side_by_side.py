"""Operands of the feed-forward operators side by side in one buffer: columns
of rows of one pitch share no element, so an output may lie beside an input;
one column further it is refused."""
import pytest
import torch

import tiled_fp32_gemm_gb300 as mt
from tiled_fp32_gemm_gb300 import build as mt_build

HAS_GPU = torch.cuda.is_available()
BASE = 0x100000


@pytest.fixture(scope="module", autouse=True)
def built_library():
    mt_build.build()
    return mt.lib()


def norm(x, y, h, rows=4, d=16, pitch=64, **change):
    """x, y and h at columns of one bf16 buffer of `pitch` columns."""
    a = mt.mt_rms_norm_args(rows=rows, d=d, x=BASE + 2 * x, ldx=pitch, residual=0x900000, ldr=d,
                            h=BASE + 2 * h, ldh=pitch, y=BASE + 2 * y, ldy=pitch, eps=1e-6,
                            dtype=mt.MT_DTYPE_BF16, out_dtype=mt.MT_DTYPE_BF16)
    for k, v in change.items():
        setattr(a, k, v)
    return mt.mt_rms_norm(a)


@pytest.mark.skipif(HAS_GPU, reason="made-up addresses")
@pytest.mark.parametrize("x,y,h", [(0, 16, 32), (48, 0, 16), (16, 32, 0), (0, 48, 16),
                                   (0, 16, 64 * 2 + 32), (64 * 3, 16, 32), (24, 40, 0)])
def test_columns_beside_one_another_are_taken(x, y, h):
    assert norm(x, y, h) == mt.MT_ERR_NO_DEVICE


@pytest.mark.parametrize("x,y,h", [(0, 15, 32), (0, 49, 24), (16, 1, 40), (0, 16, 31),
                                   (64, 15, 32), (0, 64 * 2 + 1, 32), (48, 0, 47)])
def test_columns_that_share_an_element_are_refused(x, y, h):
    assert norm(x, y, h) == mt.MT_ERR_ALIAS


def test_other_pitches_go_by_their_spans():
    assert norm(0, 16, 32, ldy=32) == mt.MT_ERR_ALIAS
    # 8-bit y of half the pitch in bytes: no column is sure to stay beside x.
    assert norm(0, 32, 1 << 16, out_dtype=mt.MT_DTYPE_E4M3, scale=0x980000,
                ldy=64) == mt.MT_ERR_ALIAS


@pytest.mark.skipif(HAS_GPU, reason="made-up addresses")
def test_pitches_count_in_bytes():
    """8-bit y in the second half of rows of 128 bytes, x in the first."""
    assert norm(0, 32, 1 << 16, out_dtype=mt.MT_DTYPE_E4M3, scale=0x980000,
                ldy=128) == mt.MT_ERR_NO_DEVICE


@pytest.mark.gpu
@pytest.mark.parametrize("d,gap", [(64, 0), (40, 1), (1001, 0), (2056, 3)])
def test_results_beside_their_operands(d, gap):
    g = torch.Generator(device="cuda").manual_seed(d)
    rows, n = 37, d + gap
    buf = torch.randn(rows, 4 * n, generator=g, device="cuda").half()
    x, r, y, h = (buf[:, i * n:i * n + d] for i in range(4))
    w = torch.randn(d, generator=g, device="cuda")

    def apart(t):
        """The same view (pitch and alignment) in a copy of the buffer."""
        return torch.as_strided(buf.clone(), t.shape, t.stride(), t.storage_offset())

    want = mt.rms_norm(apart(x), w, residual=apart(r), out=apart(y), h_out=apart(h))
    kept = buf.clone()
    got = mt.rms_norm(x, w, residual=r, out=y, h_out=h)
    assert got[0] is y and got[1] is h
    for i in range(3):
        assert torch.equal(got[i], want[i])
    want = mt.rms_norm_backward(apart(x), apart(h), w, got[2], dh=apart(r), out=apart(y))[0]
    assert torch.equal(mt.rms_norm_backward(x, h, w, got[2], dh=r, out=y)[0], want)
    b = torch.randn(d, d, generator=g, device="cuda").half()
    want = mt.linear(apart(x), b, residual=apart(r), activation="silu", out=apart(h))
    assert torch.equal(mt.linear(x, b, residual=r, activation="silu", out=h), want)
    # Nothing outside the outputs was written.
    for i, t in enumerate((x, r)):
        assert torch.equal(t, kept[:, i * n:i * n + d])
    for i in range(4):
        assert torch.equal(buf[:, i * n + d:(i + 1) * n], kept[:, i * n + d:(i + 1) * n])
