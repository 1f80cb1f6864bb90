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


@pytest.mark.parametrize("mode,gs", [(R.TOKEN_HEAD, 32), (R.MX, 16), (R.MX, 32)])
@pytest.mark.parametrize("hq", [4, 4 * LONG])
def test_large_e5m2_scales_beside_small_ones(F, mode, gs, hq):  # noqa: F811
    """Tokens whose scales are 2^10 times their neighbours', in every group of 32: rows
    that mask them keep the precision that E5M2 leaves them.

    The bound, with S the largest scale (a request's largest small one, top, times
    2^10) and rho the smallest over the largest of a group: K^ and V^ are held in units
    that put S between 1/2 and 1, and a scale is split into two f16 halves, off by at
    most 2^-25: 2^-24 / rho relative to the token (MX scales: exact).  A product below
    the normal range is off by 2^-25 more: 2^-24 S in V^, which with the term of P is W
    for that S, and sm sum |q| 2^-24 S in a score, which is F for it."""
    up, win = 10, 4
    b = Batch([90, 40], [60, 33], hq, 2, 128, 16, R.E5M2, mode, gs, seed=42, qgain=0.01,
              reach=REACH)
    out, A, Z, B, W, Fl = b.ref(device=DEV, window=win)
    *_, vscale, kscale = b.values()
    huge = [7, 37, 50, 75]
    for r in range(2):
        for j in [j for j in huge if j < b.lens[r]]:
            for sc in b.cache[2:]:
                row = sc[int(b.bt[r, j // 16]), :, j % 16]
                if mode == R.MX:
                    row += up
                else:
                    row *= 2.0 ** up
    rho = min(float(x[x > 0].min() / x.max()) for x in (vscale, kscale)) * 2.0 ** -up
    rel = 0.0 if mode == R.MX else 2.0 ** -24 / rho
    ref = (out, A, Z, B, 2.0 ** up * W + rel * A, 2.0 ** up * Fl + rel * Z)
    got = b.run(F, window=win)
    keep = []
    for r in range(2):
        for i in range(b.chunks[r]):
            pos = b.lens[r] - b.chunks[r] + i
            if not any(pos - win < j <= pos for j in huge):
                keep.append(int(b.offsets[r]) + i)
    R.check(got[keep], tuple(x[keep] for x in ref), 128, half=mode)
    assert F.get_device_error() == 0
