"""Keeping accepted paths beside rows that share pages: with the pages' counts a request that
would write to another's page is left as it was, and told."""
import ctypes

import numpy as np
import pytest
import torch

from pages_ref import SHARED, Pool
from test_gpu_pages import F, arrays, device, i32, same  # noqa: F401
from test_pages_refusals import FAKE, P, lib  # noqa: F401


@pytest.mark.parametrize("want,kw", [
    (-1, dict(ref=None)), (0, dict(ref=None, B=0)), (-1, dict(acc=None)), (-3, dict(ma=0)),
    (-4, dict(nl=P(0x4000)))])
def test_status_codes(lib, want, kw):  # noqa: F811
    ptrs, sizes = (P * 2)(0x1000, 0x2000), (ctypes.c_longlong * 2)(2048, 128)
    a = dict(acc=FAKE, ma=4, B=3, ref=FAKE, nl=P(0x8000))
    a.update(kw)
    assert lib.fp8pa_kv_keep_accepted_counted(
        a["acc"], a["ma"], FAKE, FAKE, 4, P(0x4000), a["B"], a["ref"], ctypes.cast(ptrs, P),
        ctypes.cast(sizes, P), 2, 2, 8, 16, a["nl"], None) == want


@pytest.mark.gpu
@pytest.mark.parametrize("path,moves", [([1, 3], True), ([0, 1, 2], False), ([0, 17], True),
                                        ([], False)])
def test_a_row_forked_between_its_draft_and_its_verification(F, path, moves):  # noqa: F811
    """Rows 0 and 1 hold trees of 24 nodes behind 40 and 20 tokens; row 0 was forked to row 2
    meanwhile, so that the tree's first pages are row 2's as well."""
    rng = np.random.default_rng(1)
    host, dev = arrays(rng, 20, 2, 16, [128, 4])
    p = Pool(3, 6, 20, 16, host).fill(rng, [64, 44])
    p.fork([0], [2])
    for x, d in zip(host, dev):
        d.copy_(torch.from_numpy(x))
    acc = np.full((3, 5), -1, np.int32)
    acc[0, :len(path)] = path
    acc[1, :4] = [2, 3, 5, 23]
    off = [0, 24, 48, 48]
    t, n, r = device(p)
    new = F.kv_keep_accepted(i32(acc), i32(off), t, n, F.KvPages(dev), ref_counts=r)
    if moves:  # left as it was: keeping the whole tree is what the reference calls that
        left = acc.copy()
        left[0] = -1
        want = p.keep(left, off)
        want[0] = p.n[0]
        p.flags |= SHARED
    else:
        want = p.keep(acc, off)
    assert np.array_equal(new.cpu().numpy(), want)
    same(F, p, (t, n, r), dev)


@pytest.mark.gpu
def test_shared_pages_that_are_not_written_do_not_count(F):  # noqa: F811
    """The full pages ahead of the tree are another row's, too, and so is a page that the path
    only comes from; a page outside the pool has no count.  A path of more than 32 nodes."""
    rng = np.random.default_rng(2)
    host, dev = arrays(rng, 30, 2, 16, [64, 4])
    p = Pool(3, 10, 30, 16, host).fill(rng, [32 + 100, 32 + 100])
    p.r[p.t[0, [0, 1, 7, 8]]] += 1
    acc = np.full((3, 50), -1, np.int32)
    acc[0, :40] = [*range(1, 40), 90]  # into pages 2 to 4, the last from page 7
    acc[1, :40] = range(2, 42)
    p.r[p.t[1, 4]] = 2               # the last nodes of the path: page 4 of row 1
    off = [0, 100, 200, 200]
    t, n, r = device(p)
    new = F.kv_keep_accepted(i32(acc), i32(off), t, n, F.KvPages(dev), ref_counts=r)
    acc[1] = -1
    want = p.keep(acc, off)
    want[1] = p.n[1]
    p.flags |= SHARED
    assert np.array_equal(new.cpu().numpy(), want)
    same(F, p, (t, n, r), dev)


@pytest.mark.gpu
def test_counts_that_are_not_the_pools(F):  # noqa: F811
    rng = np.random.default_rng(3)
    _, dev = arrays(rng, 20, 2, 16, [64])
    p = Pool(1, 2, 20, 16).fill(rng, [20])
    t, n, r = device(p)
    args = (i32([[1]]), i32([0, 4]), t, n, F.KvPages(dev))
    with pytest.raises(ValueError):
        F.kv_keep_accepted(*args, ref_counts=r[:19])
    with pytest.raises(TypeError):
        F.kv_keep_accepted(*args, ref_counts=r.long())
