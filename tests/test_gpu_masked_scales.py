"""Scales of masked tokens that no finite value goes with."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_gpu_prefill import DEV, F, LONG, REACH, Batch  # noqa: F401

pytestmark = pytest.mark.gpu

FLT_MAX = float(np.finfo(np.float32).max)
# scales whose largest code passes fp32, and the MX exponents of such scales
KINDS = [(R.E4M3, R.TOKEN_HEAD, 1e37), (R.E4M3, R.TOKEN_HEAD, FLT_MAX),
         (R.E5M2, R.TOKEN_HEAD, 1e37), (R.E5M2, R.TOKEN_HEAD, FLT_MAX),
         (R.INT8, R.TOKEN_HEAD, 1e37), (R.INT8, R.TOKEN_HEAD, FLT_MAX),
         (R.E4M3, R.MX, 247), (R.E4M3, R.MX, 255), (R.E5M2, R.MX, 240), (R.E5M2, R.MX, 255)]


@pytest.mark.parametrize("fmt,mode,scale", KINDS)
@pytest.mark.parametrize("which", ["k", "v", "both"])
@pytest.mark.parametrize("hq", [8, LONG * 2])  # converted by each row block, and once
def test_scales_beyond_every_finite_value(F, fmt, mode, scale, which, hq):  # noqa: F811
    """Rows that mask such tokens are as if they held anything else; rows that see such
    a V are not finite.  (Such a K gives scores of either sign, and one far below the
    others has no weight.)"""
    lens, chunks, win = [70, 50, 33, 17], [9, 50, 1, 4], 20
    b = Batch(lens, chunks, hq, 2, 128, 16, fmt, mode, 32, seed=33, reach=REACH)
    mods = dict(window=win, prefix=[5, 0, 2, 0])
    ref = b.ref(**mods)
    last = []
    for r, L in enumerate(lens):
        first = L - chunks[r] - win + 1  # the first query's window
        last.append(int(b.offsets[r + 1]) - 1)
        for j in range(L):
            # unseen by all, or the last token: seen by the last query alone
            if j != L - 1 and not (j < first and j >= mods["prefix"][r]):
                continue
            for t, sc in (("k", b.cache[2]), ("v", b.cache[3])):
                if which in (t, "both"):
                    sc[int(b.bt[r, j // 16]), :, j % 16] = scale
    got = b.run(F, **mods)
    keep = [i for i in range(int(b.offsets[-1])) if i not in last]
    R.check(got[keep], tuple(x[keep] for x in ref), 128, half=mode)
    if which != "k":
        assert not torch.isfinite(got[last]).flatten(2).all(-1).any()
    assert F.get_device_error() == 0
