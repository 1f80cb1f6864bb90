"""Score caps at the ends of fp32's range."""
import numpy as np
import pytest
import torch

import serving_ref as R
import test_gpu_decode_mod as D
from test_gpu_prefill import DEV, F, LONG, Batch, slopes_of  # noqa: F401

pytestmark = pytest.mark.gpu

FLT_MAX = float(np.finfo(np.float32).max)
# a caller's "no cap"; around the places where cap log2(e), 2 / cap and 1 / cap
# leave fp32's normal range; the smallest numbers
CAPS = [65.0, 1e33, 1e37, 2.3e38, 2.4e38, FLT_MAX, 1e-30, 1e-37, 1e-38, 1e-42, 1.4e-45]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("gain", [0.1, 30.0])
@pytest.mark.parametrize("bias", [False, True])
def test_caps_of_the_prefill(F, cap, gain, bias):  # noqa: F811
    mods = {"slopes": slopes_of(4)} if bias else {}
    Batch([77, 5, 300], [20, 5, 9], 4, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=34,
          qgain=gain).check(F, cap=cap, **mods)


@pytest.mark.parametrize("cap", CAPS)
def test_caps_over_ready_tiles(F, cap):  # noqa: F811
    b = Batch([300, 17], [60, 17], LONG, 1, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=35, reach=320)
    ref = b.ref(device=DEV, cap=cap)
    R.check(b.run(F, cap=cap), ref, 64, half=R.TOKEN_HEAD, cap=cap)


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("gain", [0.1, 30.0])
@pytest.mark.parametrize("bias", [False, True])
def test_caps_of_the_decode(F, cap, gain, bias):  # noqa: F811
    mods = {"slopes": D.slopes_of(4)} if bias else {}
    s = D.setup([77, 5, 300], 4, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=36, qgain=gain)
    D.both(F, s, 2, 128, 128 ** -0.5, R.E4M3, R.TOKEN_HEAD, cap=cap, **mods)


@pytest.mark.parametrize("cap", [1e-42, FLT_MAX])
def test_a_scale_factor_of_zero_under_extreme_caps(F, cap):  # noqa: F811
    b = Batch([70, 20], [30, 20], 4, 2, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=37)
    b.sm = 0.0
    b.check(F, cap=cap)
    s = D.setup([77, 5, 300], 4, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=38)
    D.both(F, s, 2, 128, 0.0, R.E4M3, R.TOKEN_HEAD, cap=cap)
