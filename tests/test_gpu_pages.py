"""The page operators against the references of pages_ref.py: tables, lengths, counts,
error bits and every byte of every array."""
import copy

import numpy as np
import pytest
import torch

from pages_ref import BLOCK, LEN, NO_BLOCK, OFFSETS, ROW, SHARED, TREE, Pool

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def F():
    import fp8_quantised_paged_gb300 as F
    torch.cuda.set_device(0)
    F.get_device_error()
    return F


def arrays(rng, nb, hkv, bs, kinds):
    """Arrays of random bytes: (row bytes, dtype) of each; the reference's copies and the
    device's."""
    out = [rng.integers(0, 256, (nb, hkv, bs, k), dtype=np.uint8) for k in kinds]
    return out, [torch.from_numpy(x.copy()).to(DEV) for x in out]


def device(p):
    return tuple(torch.from_numpy(x.copy()).to(DEV) for x in (p.t, p.n, p.r))


def i32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).to(DEV)


def same(F, p, got, arrays=()):
    for name, want, have in zip(("tables", "lens", "refs"), (p.t, p.n, p.r), got):
        assert np.array_equal(want, have.cpu().numpy()), name
    for i, (want, have) in enumerate(zip(p.arrays, arrays)):
        assert np.array_equal(want, have.cpu().numpy()), f"array {i}"
    assert F.get_device_error() == p.flags


# ------------------------------------------------------------------ accepted paths
# rows of a code's head dims, of scales per token, groups and blocks, of odd bytes
KINDS = {"codes": [128, 128, 4, 4], "d64 mx": [64, 64, 2, 4], "latent": [576, 36], "odd": [7, 1, 48]}


@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("bs,hkv", [(16, 8), (32, 1), (64, 3)])
def test_keep_paths(F, kinds, bs, hkv):
    rng = np.random.default_rng(bs + hkv)
    nodes = [0, 1, 2, 5, 8, 40, 77, 64]
    ctx = [3, 0, bs - 1, bs, 2 * bs - 3, 5, 100, 0]
    lens = [c + n for c, n in zip(ctx, nodes)]
    cols = max(lens) // bs + 2
    nb = sum(-(-n // bs) for n in lens) + 2
    host, dev = arrays(rng, nb, hkv, bs, KINDS[kinds])
    p = Pool(len(lens), cols, nb, bs, host).fill(rng, lens)
    acc = np.full((len(lens), 70), -1, np.int32)
    acc[1, 0] = 0
    acc[2, :1] = 1                      # one row moves by one
    acc[3, :3] = [1, 3, 4]              # a moved row is another's place
    acc[4, :8] = range(8)               # all kept: nothing moves
    acc[5, :39] = range(1, 40)          # every row moves by one, over more than 32 places
    acc[6, :70] = range(7, 77)          # as long as the array: no end mark
    acc[7, :4] = [0, 2, 33, 63]
    off = np.concatenate([[0], np.cumsum(nodes)])
    t, n, r = device(p)
    new = F.kv_keep_accepted(i32(acc), i32(off), t, n, F.KvPages(dev))
    want = p.keep(acc, off)
    assert p.flags == 0
    assert np.array_equal(new.cpu().numpy(), want)
    same(F, p, (t, n, r), dev)


@pytest.mark.parametrize("path,n,flag", [
    ([2, 1, 3], 5, TREE), ([0, 0, 1], 5, TREE), ([0, 5], 5, TREE), ([7], 5, TREE),
    ([2 ** 31 - 1], 5, TREE), ([1, -7, 9], 5, 0), ([-1, 2], 5, 0), ([0], 0, TREE)])
def test_keep_cuts_a_path_at_its_first_bad_node(F, path, n, flag):
    rng = np.random.default_rng(1)
    host, dev = arrays(rng, 6, 2, 16, [64, 4])
    p = Pool(2, 3, 6, 16, host).fill(rng, [20, 17 + n])
    acc = np.full((2, 4), -1, np.int32)
    acc[0, :2] = [1, 2]
    acc[1, :len(path)] = path
    off = [0, 4, 4 + n]
    t, ln, r = device(p)
    new = F.kv_keep_accepted(i32(acc), i32(off), t, ln, F.KvPages(dev))
    assert np.array_equal(new.cpu().numpy(), p.keep(acc, off))
    assert p.flags == flag
    same(F, p, (t, ln, r), dev)


def test_keep_leaves_bad_requests_alone(F):
    rng = np.random.default_rng(2)
    host, dev = arrays(rng, 12, 2, 16, [64, 4])
    p = Pool(6, 3, 12, 16, host).fill(rng, [20, 20, 20, 20, 20, 20])
    p.t[4, 1] = -1     # a moved row's page is missing
    p.t[5, 1] = 12     # or outside the pool
    p.n[1] = 49        # longer than its table
    p.n[2] = 3         # shorter than its tree
    acc = np.tile(np.array([1, 3, -1, -1], np.int32), (6, 1))
    acc[4:] = [1, 4, 5, 6]
    for off, flag in (([0, 6, 12, 18, 24, 31, 38], LEN | BLOCK),
                      ([0, -6, 12, 18, 16, 23, 30], LEN | BLOCK | OFFSETS)):
        q, dv = copy.deepcopy(p), [x.clone() for x in dev]
        t, ln, r = device(q)
        new = F.kv_keep_accepted(i32(acc), i32(off), t, ln, F.KvPages(dv))
        assert np.array_equal(new.cpu().numpy(), q.keep(acc, off))
        assert q.flags == flag
        same(F, q, (t, ln, r), dv)


# ------------------------------------------------------------------ forks
def test_fork_shares_full_pages_and_copies_the_last(F):
    rng = np.random.default_rng(3)
    for bs, hkv in ((16, 8), (32, 3), (64, 1)):
        host, dev = arrays(rng, 60, hkv, bs, [128, 64, 4])
        seg = rng.integers(0, 2 ** 31, (60, 4)).astype(np.int32)  # page scales: no row per token
        p = Pool(20, 6, 60, bs, host + [seg]).fill(rng, [0, 1, bs - 1, bs, bs + 1, 3 * bs, 5 * bs + 7])
        dev = dev + [torch.from_numpy(seg.copy()).to(DEV)]
        src = [1, 2, 3, 4, 5, 6, 0, 6, 6, 1]
        dst = [19, 7, 9, 8, 10, 18, 17, 11, 12, 13]
        t, n, r = device(p)
        F.kv_fork(i32(src), i32(dst), t, n, r, F.KvPages(dev))
        p.fork(src, dst)
        assert p.flags == 0
        same(F, p, (t, n, r), dev)


def test_forks_that_cannot_be_made(F):
    rng = np.random.default_rng(4)
    host, dev = arrays(rng, 20, 2, 16, [64])
    p = Pool(12, 4, 20, 16, host).fill(rng, [20, 33, 16, 40, 0, 0, 0, 0, 0, 0, 0, 20])
    p.t[3, 2] = 20     # a last page outside the pool
    p.n[11] = 65       # longer than its table
    # rows outside the tables, onto itself, onto a row that is not empty, a row wanted
    # twice (the first gets it), a source that another fork fills (empty, as before)
    src = [0, -1, 12, 1, 2, 0, 1, 4, 3, 11, 1]
    dst = [4, 5, 5, 12, 2, 1, 4, 6, 7, 8, 9]
    t, n, r = device(p)
    F.kv_fork(i32(src), i32(dst), t, n, r, F.KvPages(dev))
    p.fork(src, dst)
    assert p.flags == ROW | BLOCK | LEN
    same(F, p, (t, n, r), dev)


def test_fork_without_free_pages(F):
    rng = np.random.default_rng(5)
    host, dev = arrays(rng, 8, 2, 16, [64])
    p = Pool(10, 2, 8, 16, host).fill(rng, [20, 16, 17, 10])  # two pages are free
    src, dst = [0, 2, 1, 3], [4, 5, 6, 7]
    t, n, r = device(p)
    F.kv_fork(i32(src), i32(dst), t, n, r, F.KvPages(dev))
    p.fork(src, dst)
    assert p.flags == NO_BLOCK and list(p.n[4:8]) == [20, 17, 16, 0]
    same(F, p, (t, n, r), dev)


def test_many_forks_over_many_arrays(F):
    """More forks than a planning step takes, more arrays than a launch takes."""
    rng = np.random.default_rng(6)
    rows, nb = 1400, 3000
    host, dev = arrays(rng, nb, 1, 16, [1] * 131)
    lens = np.zeros(rows, np.int64)
    lens[:60] = rng.integers(1, 80, 60)
    p = Pool(rows, 5, nb, 16, host).fill(rng, lens)
    dst = rng.permutation(np.arange(60, rows))[:1300]
    src = rng.integers(0, 60, 1300)
    t, n, r = device(p)
    F.kv_fork(i32(src), i32(dst), t, n, r, F.KvPages(dev))
    p.fork(src, dst)
    same(F, p, (t, n, r), dev)
    acc = np.full((rows, 2), -1, np.int32)
    acc[:, 0] = 1
    off = np.arange(rows + 1) * 2
    p.n[p.n == 0], p.n[p.n == 1] = 2, 2
    p.t[p.t < 0] = nb - 1
    t, n, r = device(p)
    # rows that share pages write alike only if they move alike: one row at a time is kept
    acc[1:, 0] = -1
    new = F.kv_keep_accepted(i32(acc), i32(off), t, n, F.KvPages(dev))
    assert np.array_equal(new.cpu().numpy(), p.keep(acc, off))
    same(F, p, (t, n, r), dev)


# ------------------------------------------------------------------ resizing
def test_resize_grows_shrinks_and_frees(F):
    rng = np.random.default_rng(7)
    for rows, nb, bs, top in ((7, 40, 16, 90), (300, 3000, 32, 400), (2100, 40000, 64, 2000)):
        cols = top // bs + 2
        p = Pool(rows, cols, nb, bs).fill(rng, rng.integers(0, top // 3, rows) * (rng.random(rows) < .8))
        for step in range(3):
            then = np.where(rng.random(rows) < .5, p.n + rng.integers(0, 3, rows),
                            rng.integers(0, top // 2, rows) * (rng.random(rows) < .8))
            t, n, r = device(p)
            F.kv_resize(i32(then), t, n, r, bs)
            p.resize(then)
            same(F, p, (t, n, r))
            p.flags = 0


def test_resize_without_free_pages(F):
    rng = np.random.default_rng(8)
    p = Pool(6, 8, 12, 16).fill(rng, [16, 32, 48, 0, 20, 5])  # 9 pages held
    # row 1 gives two back: 5 are free; row 0 takes 2, row 2 does not fit, and those
    # behind it wait with it, though row 4 would fit; row 5 keeps its one page
    then = [48, 0, 120, 16, 33, 9]
    t, n, r = device(p)
    F.kv_resize(i32(then), t, n, r, 16)
    p.resize(then)
    assert p.flags == NO_BLOCK and list(p.n) == [48, 0, 48, 0, 20, 9]
    same(F, p, (t, n, r))


def test_resize_keeps_off_shared_pages(F):
    rng = np.random.default_rng(9)
    p = Pool(6, 6, 40, 16).fill(rng, [50, 64])
    p.fork([0, 1, 1], [2, 3, 4])
    # 0 cut inside a page of 2's; 1 cut between pages; 2 grows in its own last page; 3 freed;
    # 4 cut inside a page that 1 and 3 give up in the same call: still refused
    then = [40, 32, 53, 0, 50, 0]
    t, n, r = device(p)
    F.kv_resize(i32(then), t, n, r, 16)
    p.resize(then)
    assert p.flags == SHARED and list(p.n) == [50, 32, 53, 0, 64, 0]
    same(F, p, (t, n, r))
    # a partly filled page that was shared by hand is not grown in
    p.flags = 0
    p.t[5, :4], p.n[5] = p.t[0, :4], 50
    p.r[p.t[0, :4]] += 1
    then = [51, 32, 53, 0, 64, 50]
    t, n, r = device(p)
    F.kv_resize(i32(then), t, n, r, 16)
    p.resize(then)
    assert p.flags == SHARED and p.n[0] == 50
    same(F, p, (t, n, r))


def test_resize_with_bad_lengths_and_pages(F):
    rng = np.random.default_rng(10)
    p = Pool(5, 3, 20, 16).fill(rng, [20, 20, 48, 20, 0])
    p.n[0] = 49
    p.t[2, 1] = -5
    t, n, r = device(p)
    then = [10, -1, 0, 49, 48]
    F.kv_resize(i32(then), t, n, r, 16)
    p.resize(then)
    assert p.flags == LEN | BLOCK
    same(F, p, (t, n, r))
    F.kv_resize(n, t, n, r, 16)  # the lengths themselves: nothing changes but the bad row's bit
    p.flags = LEN
    same(F, p, (t, n, r))


# ------------------------------------------------------------------ compacting
@pytest.mark.parametrize("rows,nb,bs,top", [(1, 1, 16, 16), (1, 2, 16, 16), (3, 33, 64, 200),
                                            (40, 301, 16, 90), (64, 2000, 32, 300),
                                            (500, 20001, 16, 600)])
def test_compact(F, rows, nb, bs, top):
    rng = np.random.default_rng(nb)
    host, dev = arrays(rng, nb, 2 if nb < 5000 else 1, bs, [64, 4])
    seg = rng.integers(0, 2 ** 31, (nb, 4)).astype(np.int32)
    lens = rng.integers(0, top + 1, rows)
    while sum(-(-int(n) // bs) for n in lens) > nb:
        lens //= 2
    p = Pool(rows + 3, top // bs + 1, nb, bs, host + [seg]).fill(rng, lens)
    if rows > 3:
        p.fork([0, 1, 2], [rows, rows + 1, rows + 2])
        p.r[rng.permutation(nb)[:5]] += 1  # pages that the caller keeps
    for x, d in zip(host, dev):
        d.copy_(torch.from_numpy(x))
    dev = dev + [torch.from_numpy(seg.copy()).to(DEV)]
    t, n, r = device(p)
    got = F.kv_compact(t, n, r, F.KvPages(dev))
    want = p.compact()
    assert p.flags == 0
    assert np.array_equal(got.cpu().numpy(), want)
    same(F, p, (t, n, r), dev)
    again = F.kv_compact(t, n, r, F.KvPages(dev))  # nothing is left to move
    assert np.array_equal(again.cpu().numpy(), p.compact())
    same(F, p, (t, n, r), dev)


def test_compact_empty_and_full_pools(F):
    rng = np.random.default_rng(11)
    for lens in ([0, 0], [32, 16]):
        host, dev = arrays(rng, 3, 1, 16, [64])
        p = Pool(2, 2, 3, 16, host).fill(rng, lens)
        t, n, r = device(p)
        got = F.kv_compact(t, n, r, F.KvPages(dev))
        assert np.array_equal(got.cpu().numpy(), p.compact())
        same(F, p, (t, n, r), dev)


def test_compact_leaves_bad_entries(F):
    rng = np.random.default_rng(12)
    host, dev = arrays(rng, 30, 1, 16, [64])
    p = Pool(4, 4, 30, 16, host).fill(rng, [30, 60, 20, 10])
    p.t[0, 0], p.t[1, 1] = 30, int(np.flatnonzero(p.r == 0)[0])
    p.n[2] = -1
    t, n, r = device(p)
    got = F.kv_compact(t, n, r, F.KvPages(dev))
    assert np.array_equal(got.cpu().numpy(), p.compact())
    assert p.flags == BLOCK | LEN
    same(F, p, (t, n, r), dev)


# ------------------------------------------------------------------ streams and graphs
def test_a_round_of_calls_captured_and_replayed(F):
    """Grow, keep, shrink, fork, free and compact in one graph, replayed on new states, on a
    stream of its own."""
    rng = np.random.default_rng(13)
    host, dev = arrays(rng, 80, 2, 16, [128, 4])
    pages = F.KvPages(dev)
    first = Pool(12, 6, 80, 16, host).fill(rng, [50, 17, 32, 5, 0, 60])
    t, n, r = device(first)
    acc, off = i32(np.full((12, 3), -1)), i32(np.zeros(13))
    then, less, src, dst = i32(np.zeros(12)), i32(np.zeros(12)), i32([0, 1, 5]), i32([6, 7, 8])
    side = torch.cuda.Stream()

    def calls():
        F.kv_resize(then, t, n, r, 16)
        kept = F.kv_keep_accepted(acc, off, t, n, pages)
        F.kv_resize(kept, t, n, r, 16)
        F.kv_fork(src, dst, t, n, r, pages)
        F.kv_resize(less, t, n, r, 16)
        return F.kv_compact(t, n, r, pages)

    with torch.cuda.stream(side):
        calls()
        side.synchronize()
        F.get_device_error()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            moved = calls()
    for seed in range(4):
        rng = np.random.default_rng(100 + seed)
        p = Pool(12, 6, 80, 16, [rng.integers(0, 256, x.shape, dtype=np.uint8) for x in host])
        p.fill(rng, np.concatenate([rng.integers(0, 60, 6), np.zeros(6, np.int64)]))
        nodes = rng.integers(0, 9, 12) * (np.arange(12) < 6)
        a = np.full((12, 3), -1, np.int32)
        for b in range(6):
            k = min(3, int(nodes[b]))
            a[b, :k] = np.sort(rng.permutation(nodes[b])[:k])
        o = np.concatenate([[0], np.cumsum(nodes)])
        m = (p.n + nodes) * (np.arange(12) < 6)
        for d, h in zip((t, n, r, acc, off, then, *dev), (p.t, p.n, p.r, a, o, m, *p.arrays)):
            d.copy_(torch.from_numpy(np.ascontiguousarray(h)))
        p.resize(m)
        p.resize(p.keep(a, o))
        p.fork([0, 1, 5], [6, 7, 8])
        z = np.where(np.arange(12) < 4, p.n, 0)
        less.copy_(torch.from_numpy(z.astype(np.int32)))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay()
        torch.cuda.synchronize()
        p.resize(z)
        want = p.compact()
        assert p.flags == 0
        assert np.array_equal(moved.cpu().numpy(), want), seed
        same(F, p, (t, n, r), dev)
