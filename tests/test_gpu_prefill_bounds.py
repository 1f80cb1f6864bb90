"""What the prefill leaves alone: rows of skipped requests, and memory behind its own."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_gpu_prefill import DEV, F, REACH, Batch  # noqa: F401

pytestmark = pytest.mark.gpu

KEPT = 7.0


@pytest.mark.parametrize("hq", [4, 1536])  # converted by each row block, and once
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offsets,skipped", [
    ([0, 9, 6], (0, 1)), ([-1, 4, 6], (0,)), ([0, 4, 7], (1,)), ([5, 2, 6], (0,)),
    ([0, 3, 2 ** 31 - 1], (1,)), ([-2 ** 31, 0, 6], (0,))])
def test_bad_offsets_skip_their_request_alone(F, hq, dt, offsets, skipped):  # noqa: F811
    """Two requests of 6 rows in all: a skipped one's rows stay, its neighbour is right."""
    from fp8_quantised_paged_gb300 import _native as N
    total, guard = 6, 40
    b = Batch([20, 30], [4, 2], hq, 1, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=41, reach=REACH)
    b.offsets = np.array(offsets, np.int32)
    buf = torch.full((total + guard, hq, 64), KEPT, dtype=dt, device=DEV)
    out = buf[guard // 2:guard // 2 + total]
    assert b.run(F, out=out, out_dtype=dt) is out
    assert F.get_device_error() == N.DEVERR_Q_OFFSETS
    good = [r for r in (0, 1) if r not in skipped]
    rows = [i for r in good for i in range(offsets[r], offsets[r + 1])]
    own = np.array([0, 0, 0], np.int32)
    for r in good:  # the reference over the good requests alone
        own[:] = [offsets[1], offsets[1], offsets[1]]
        own[r], own[r + 1] = offsets[r], offsets[r + 1]
        b.offsets = own
        ref = b.ref(device=DEV)
        R.check(out[rows], tuple(x[rows] for x in ref), 64, bf16=dt == torch.bfloat16,
                half=R.TOKEN_HEAD)
    left = [i for i in range(total) if i not in rows]
    assert (out[left] == KEPT).all()
    assert (buf[:guard // 2] == KEPT).all() and (buf[guard // 2 + total:] == KEPT).all()
