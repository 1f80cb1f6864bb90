"""Windows up to the largest int and beyond: as wide as any context, so none at all."""
import pytest
import torch

import serving_ref as R
import test_gpu_decode_mod as D
from test_gpu_prefill import DEV, F, LONG, REACH, Batch  # noqa: F401

pytestmark = pytest.mark.gpu

WIDE = [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 31 - 40, 2 ** 31, 2 ** 32 + 5, 2 ** 63 - 1]


@pytest.mark.parametrize("window", WIDE)
@pytest.mark.parametrize("hq", [8, LONG * 2])
@pytest.mark.parametrize("prefix", [None, [3, 0, 200]])
def test_wide_windows_of_the_prefill(F, window, hq, prefix):  # noqa: F811
    b = Batch([130, 17, 200], [100, 17, 64], hq, 2, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=49,
              reach=REACH)
    want = b.run(F, prefix=prefix)
    assert torch.equal(b.run(F, window=window, prefix=prefix), want)
    assert F.get_device_error() == 0


@pytest.mark.parametrize("window", WIDE)
@pytest.mark.parametrize("hq", [8, LONG * 2])
def test_wide_windows_over_chunks_longer_than_their_requests(F, window, hq):  # noqa: F811
    """Positions below zero: those rows see nothing, the others are as without a window."""
    from fp8_quantised_paged_gb300 import _native as N
    b = Batch([130, 40, 200], [100, 40, 64], hq, 2, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=50,
              reach=REACH)
    b.lens[0], b.lens[1], b.lens[2] = 60, 0, 9
    want = b.run(F)
    assert F.get_device_error() == N.DEVERR_SEQ_LEN
    got = b.run(F, window=window)
    assert F.get_device_error() == N.DEVERR_SEQ_LEN
    assert torch.equal(got, want)
    assert not got[:40].any() and got[40:100].any()
    assert not got[100:195].any() and got[195:].any()


@pytest.mark.parametrize("window", WIDE)
def test_wide_windows_of_the_decode(F, window):  # noqa: F811
    s = D.setup(D.LENS, 8, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=51)
    want = D.call(F, s, 2, 0.09, R.E4M3, R.TOKEN_HEAD, cap=9.0)
    assert torch.equal(D.call(F, s, 2, 0.09, R.E4M3, R.TOKEN_HEAD, cap=9.0, window=window), want)
    assert F.get_device_error() == 0


@pytest.mark.parametrize("window", [-1, -2 ** 31, -2 ** 31 - 1, -2 ** 40])
def test_negative_windows_are_refused(F, window):  # noqa: F811
    b = Batch([30], [5], 8, 2, 64, 16, R.E4M3, R.TOKEN_HEAD)
    with pytest.raises(F.Fp8paError):
        b.run(F, window=window)
    s = D.setup([30], 8, 2, 128, 16, R.E4M3, R.TOKEN_HEAD)
    with pytest.raises(F.Fp8paError):
        D.call(F, s, 2, 0.09, R.E4M3, R.TOKEN_HEAD, window=window)
