"""Rows that see a value that is not finite."""
import numpy as np
import pytest
import torch

import serving_ref as R
import test_gpu_decode_mod as D
from test_gpu_prefill import DEV, F, LONG, REACH, Batch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[1, 40], [40, 33], [900, 2]])
@pytest.mark.parametrize("what", ["k codes", "k scale", "v codes", "v scale", "q"])
@pytest.mark.parametrize("every", [True, False])
def test_a_decode_row_that_sees_nan_is_nan(F, lens, what, every):  # noqa: F811
    """In all visible tokens of request 0, or in its last."""
    s = D.setup(lens, 8, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=39)
    ref = D.reference(s, 2, 0.088, R.E4M3, R.TOKEN_HEAD, window=500)
    q, kc, vc, ks, vs, bt, _ = s
    if what == "q":
        q[0] = float("nan")
    for j in range(0 if every else lens[0] - 1, lens[0]):
        t = {"k codes": kc, "k scale": ks, "v codes": vc, "v scale": vs}.get(what)
        if t is not None:
            t[int(bt[0, j // 16]), :, j % 16] = 0x7F if "codes" in what else float("nan")
    got = D.call(F, s, 2, 0.088, R.E4M3, R.TOKEN_HEAD, window=500)
    assert not torch.isfinite(got[0]).all(-1).any()
    R.check(got[1:], tuple(x[1:] if np.ndim(x) else x for x in ref), 128)


@pytest.mark.parametrize("lens", [[1, 40], [40, 33], [900, 20]])
@pytest.mark.parametrize("what", ["k codes", "k scale", "v codes", "v scale", "q"])
@pytest.mark.parametrize("every", [True, False])
@pytest.mark.parametrize("hq", [8, LONG * 2])
def test_a_prefill_row_that_sees_nan_is_nan(F, lens, what, every, hq):  # noqa: F811
    """In all tokens of request 0, or in its last: that its last query alone sees."""
    chunks = [min(n, 10) for n in lens]
    b = Batch(lens, chunks, hq, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=40, reach=REACH)
    ref = b.ref(device=DEV)
    kc, vc, ks, vs = b.cache
    n = chunks[0]
    if what == "q":
        b.q[0 if every else n - 1:n] = float("nan")
    for j in range(0 if every else lens[0] - 1, lens[0]):
        t = {"k codes": kc, "k scale": ks, "v codes": vc, "v scale": vs}.get(what)
        if t is not None:
            t[int(b.bt[0, j // 16]), :, j % 16] = 0x7F if "codes" in what else float("nan")
    got = b.run(F)
    bad = list(range(0 if every else n - 1, n))
    keep = [i for i in range(got.shape[0]) if i not in bad]
    assert not torch.isfinite(got[bad]).all(-1).any()
    R.check(got[keep], tuple(x[keep] for x in ref), 128, half=R.TOKEN_HEAD)
