"""Resizes of rows whose last, partly filled page is missing from their table."""
import numpy as np
import pytest
import torch

from pages_ref import BLOCK, Pool
from test_gpu_pages import DEV, F, device, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("entry", [-1, -7, 40, 2 ** 31 - 1])
@pytest.mark.parametrize("then", [21, 16 * 3, 16 * 3 + 5, 18])
def test_a_row_with_a_hole_at_its_next_token_is_left(F, entry, then):  # noqa: F811
    """Growing within the missing page, past it, and ending inside it: the row and the free
    pages stay as they were, and its neighbours get theirs."""
    rng = np.random.default_rng(1)
    p = Pool(4, 5, 40, 16).fill(rng, [20, 20, 17, 33])
    p.r[p.t[1, 1]] = 0  # the page that the row no longer names is free
    p.t[1, 1] = entry
    t, n, r = device(p)
    free = p.free()
    F.kv_resize(i32([36, then, 0, 40]), t, n, r, 16)
    assert F.get_device_error() == BLOCK
    want = p.t.copy()
    free = sorted(free + [int(x) for x in p.t[2, :2]])
    want[0, 2], want[2, :2] = free[0], -1
    refs = p.r.copy()
    refs[p.t[2, :2]] = 0
    refs[free[0]] = 1
    assert n.cpu().tolist() == [36, 20, 0, 40]
    assert np.array_equal(t.cpu().numpy(), want)
    assert np.array_equal(r.cpu().numpy(), refs)


def test_a_hole_elsewhere_does_not_hold_a_row(F):  # noqa: F811
    """Behind the new length, at a page's end, and in a row that keeps its length."""
    rng = np.random.default_rng(2)
    p = Pool(4, 4, 20, 16).fill(rng, [40, 32, 20, 20])
    lost = [p.t[0, 2], p.t[1, 1], p.t[2, 1], p.t[3, 1]]
    p.t[0, 2] = p.t[1, 1] = p.t[2, 1] = p.t[3, 1] = -1
    p.r[lost] = 0
    t, n, r = device(p)
    free = p.free()
    F.kv_resize(i32([24, 33, 20, 0]), t, n, r, 16)
    assert F.get_device_error() == BLOCK  # two of them give an entry back that is none
    assert n.cpu().tolist() == [24, 33, 20, 0]
    free = sorted(free + [int(p.t[3, 0])])
    want, refs = p.t.copy(), p.r.copy()
    refs[p.t[3, 0]] = 0
    want[3, 0] = -1
    want[1, 2] = free[0]
    refs[free[0]] = 1
    assert np.array_equal(t.cpu().numpy(), want)
    assert np.array_equal(r.cpu().numpy(), refs)
    assert torch.equal(t[2], i32(p.t[2]))
