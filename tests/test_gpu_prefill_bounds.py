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


@pytest.mark.parametrize("d,fmt,mode", [(128, R.E4M3, R.TOKEN_HEAD), (64, R.INT8, R.TOKEN_HEAD),
                                        (128, R.E5M2, R.MX)])
def test_any_workspace_that_is_taken_is_not_overrun(F, d, fmt, mode):  # noqa: F811
    """Below the size function's answer tiles are converted where they are used; below
    the plan and the pieces the call is refused.  Nothing behind is written."""
    b = Batch([700, 3, 400], [300, 3, 200], 16, 2, d, 16, fmt, mode, seed=45)
    ref = b.ref(device=DEV, window=350)
    full = F.prefill_workspace_bytes(503, 3, 16, 2, d, 16, b.bt.shape[1])
    buf = torch.empty(full, dtype=torch.uint8, device=DEV)

    def run(n):
        buf.fill_(0xA5)
        got = b.run(F, window=350, workspace=buf[:n])
        assert (buf[n:] == 0xA5).all()
        R.check(got, ref, d, half=mode)
        return got

    once = run(full)
    assert torch.equal(run(full), once)
    each = run(full - 256)  # the tiles no longer fit
    low, high = 0, full - 256  # refused, taken
    while high - low > 256:
        n = (low + high) // 512 * 256
        try:
            assert torch.equal(run(n), each)
            high = n
        except F.Fp8paError as e:
            assert e.code == -5
            low = n
    assert high < full - 3 * (700 // 128) * 2 * 4 * 128 * d  # without any tile
    assert F.get_device_error() == 0


def test_a_workspace_of_a_large_batch_serves_a_small_one(F):  # noqa: F811
    """40 requests of 9 queries need no tiles, one of 300 would."""
    big = Batch([400] * 40, [9] * 40, 16, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=46)
    size = lambda b: F.prefill_workspace_bytes(  # noqa: E731
        int(b.offsets[-1]), len(b.lens), 16, 2, 128, 16, b.bt.shape[1])
    ws = torch.empty(size(big), dtype=torch.uint8, device=DEV)
    for small in (Batch([400], [300], 16, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=47),
                  Batch([4000], [300], 16, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=48), big):
        R.check(small.run(F, workspace=ws), small.ref(device=DEV), 128, half=R.TOKEN_HEAD)
    assert size(Batch([4000], [300], 16, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=48)) > size(big)
    assert F.get_device_error() == 0
