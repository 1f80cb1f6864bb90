"""Forks that want one row: the first that can be made gets it."""
import numpy as np
import pytest

from pages_ref import BLOCK, LEN, NO_BLOCK, ROW, Pool
from test_gpu_pages import F, arrays, device, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def pool(seed, nb=20):
    rng = np.random.default_rng(seed)
    host, dev = arrays(rng, nb, 2, 16, [64])
    return Pool(8, 4, nb, 16, host).fill(rng, [20, 33, 16, 40]), dev


def check(F, p, dev, src, dst, made, flags):  # noqa: F811
    """The forks of `made` alone, and these error bits."""
    t, n, r = device(p)
    F.kv_fork(i32(src), i32(dst), t, n, r, F.KvPages(dev))
    assert F.get_device_error() == flags
    p.fork([src[i] for i in made], [dst[i] for i in made])
    for want, have in zip((p.t, p.n, p.r, p.arrays[0]), (t, n, r, dev[0])):
        assert np.array_equal(want, have.cpu().numpy())


@pytest.mark.parametrize("bad", [-1, 8, 2 ** 31 - 1, 5])  # outside the tables; the row itself
def test_a_fork_without_a_source_uses_up_no_row(F, bad):  # noqa: F811
    p, dev = pool(1)
    check(F, p, dev, [bad, 0, 1, bad], [5, 5, 5, 6], [1], ROW)


def test_a_fork_of_a_bad_row_uses_up_no_row(F):  # noqa: F811
    p, dev = pool(2)
    p.n[2] = 65         # longer than its table
    p.t[3, 2] = -1      # a last page that is not there
    check(F, p, dev, [2, 0, 3, 1, 1], [5, 5, 6, 7, 6], [1, 3, 4], LEN | BLOCK)


def test_the_first_of_several_is_made(F):  # noqa: F811
    p, dev = pool(3)
    check(F, p, dev, [3, 0, 1, 2], [4, 4, 4, 7], [0, 3], ROW)


def test_a_fork_that_finds_no_page_uses_up_its_row(F):  # noqa: F811
    p, dev = pool(4, 9)  # 9 pages, all held
    assert not p.free()
    check(F, p, dev, [0, 2, 2], [4, 4, 5], [2], NO_BLOCK | ROW)


def test_claims_over_more_forks_than_a_planning_step(F):  # noqa: F811
    rng = np.random.default_rng(5)
    rows, nb = 3000, 6000
    host, dev = arrays(rng, nb, 1, 16, [16])
    p = Pool(rows, 5, nb, 16, host).fill(rng, rng.integers(1, 80, 60))
    dst = rng.integers(60, 1200, 2900)
    src = np.where(rng.random(2900) < .5, rows + 5, rng.integers(0, 60, 2900))
    made, taken = [], set()
    for i in range(2900):
        if src[i] < rows and int(dst[i]) not in taken:
            taken.add(int(dst[i]))
            made.append(i)
    assert max(made) > 1024 and len(made) < 2900
    check(F, p, dev, src.tolist(), dst.tolist(), made, ROW)
