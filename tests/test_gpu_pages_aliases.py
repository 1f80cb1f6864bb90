"""Arguments of the page operators that overlap what a call changes are refused; real tensors,
so that a call that is made all the same stays within them."""
import numpy as np
import pytest
import torch

from pages_ref import Pool
from test_gpu_pages import DEV, F, arrays, device  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture()
def state():
    rng = np.random.default_rng(1)
    _, dev = arrays(rng, 40, 2, 16, [64, 4])
    p = Pool(6, 8, 40, 16).fill(rng, [20, 33, 40, 0, 0, 0])
    one = torch.zeros(200, dtype=torch.int32, device=DEV)
    one[100:112] = -1  # empty paths of empty trees
    # tables, lengths and counts in one buffer, the rest behind them
    t, n, r = one[:48].view(6, 8), one[48:54], one[54:94]
    for x, y in zip((t, n, r), device(p)):
        x.copy_(y)
    return one, t, n, r, dev


def unchanged(F, one, call):  # noqa: F811
    before = one.clone()
    with pytest.raises(F.Fp8paError):
        call()
    assert torch.equal(one, before) and F.get_device_error() == 0


def test_keep(F, state):  # noqa: F811
    one, t, n, r, dev = state
    pages = F.KvPages(dev)
    acc, off = one[100:112].view(6, 2), one[120:127]
    keep = lambda **kw: F.kv_keep_accepted(acc, off, t, n, pages, **kw)  # noqa: E731
    for bad in (n, one[49:55], off[:6], one[115:121], one[126:132], one[95:101], one[111:117],
                one[42:48], one[:6]):
        unchanged(F, one, lambda: keep(new_lens=bad))
    unchanged(F, one, lambda: keep(new_lens=one[90:96], ref_counts=r))
    for good in (one[94:100], one[112:118], one[127:133]):
        keep(new_lens=good, ref_counts=r)
    keep(new_lens=one[60:66].clone())
    assert F.get_device_error() == 0


def test_fork_resize_compact(F, state):  # noqa: F811
    one, t, n, r, dev = state
    pages = F.KvPages(dev)
    rows = one[100:102].copy_(torch.tensor([3, 4], device=DEV))
    for bad in (one[46:48], n[:2], one[53:55], r[5:7]):
        unchanged(F, one, lambda: F.kv_fork(bad, rows, t, n, r, pages))
        unchanged(F, one, lambda: F.kv_fork(rows, bad, t, n, r, pages))
    for bad in (one[43:49], one[49:55], one[93:99], r[:6]):
        unchanged(F, one, lambda: F.kv_resize(bad, t, n, r, 16))
    for bad in (one[8:48], one[50:90], r, one[93:133]):
        unchanged(F, one, lambda: F.kv_compact(t, n, r, pages, page_map=bad))
    F.kv_resize(n, t, n, r, 16)
    F.kv_compact(t, n, r, pages, page_map=one[94:134])
    assert F.get_device_error() == 0
