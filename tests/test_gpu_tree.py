"""Tree attention against the 64-bit reference of tree_ref.py: shapes, formats, scale modes,
masks, splits, bad arguments found on the device."""
import numpy as np
import pytest
import torch

from serving_ref import (E4M3, E5M2, INT8, MX, SEGMENT, STATIC, TOKEN_HEAD, chunk_values,
                         make_cache, make_tables)
from tree_ref import check_tree, tree_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def F():
    import fp8_quantised_paged_gb300 as F
    torch.cuda.set_device(0)
    F.get_device_error()
    return F


def grow(rng, n, kind):
    """Parents of n nodes: a line, candidates for one place, several roots, or any tree."""
    if kind == "line":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "roots":
        return [-1 if i < 3 else int(rng.integers(-1, i)) for i in range(n)]
    return [-1] + [int(rng.integers(max(0, i - 8), i)) for i in range(1, n)]


KINDS = ["any", "line", "star", "roots"]


class Case:
    def __init__(self, seed, ctx, nodes, hq, hkv, d, bs, fmt, mode, gs=32, window=0, prefix=None,
                 cap=0.0, alibi=False, sm=None, kinds=KINDS):
        rng = self.rng = np.random.default_rng(seed)
        self.lens = np.array([c + n for c, n in zip(ctx, nodes)], np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.parents = np.array([p for i, n in enumerate(nodes) if n
                                 for p in grow(rng, n, kinds[i % len(kinds)])], np.int32)
        self.bt, nb = make_tables(rng, self.lens, bs)
        self.cache = [x.to(DEV) for x in make_cache(rng, nb, hkv, bs, d, fmt, mode, gs)]
        total = int(self.offsets[-1])
        q = rng.standard_normal((total, hq, d)) * np.exp(rng.normal(0, .5, (total, hq, 1)))
        self.q = torch.from_numpy(q.astype(np.float32)).to(DEV).bfloat16()
        self.hq, self.hkv, self.d, self.bs, self.fmt, self.mode, self.gs = hq, hkv, d, bs, fmt, mode, gs
        self.window, self.cap = window, cap
        self.prefix = None if prefix is None else np.array(prefix, np.int32)
        self.slopes = (np.exp2(-8.0 * np.arange(1, hq + 1) / hq).astype(np.float32)
                       if alibi else None)
        self.sm = d ** -0.5 if sm is None else sm

    def args(self):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        return ((self.q, t(self.offsets), t(self.parents), *self.cache, self.bt.to(DEV),
                 t(self.lens), self.hkv, self.sm),
                dict(window=self.window, logit_cap=self.cap,
                     prefix_lens=None if self.prefix is None else t(self.prefix),
                     alibi_slopes=None if self.slopes is None else t(self.slopes), fmt=self.fmt,
                     scale_mode=self.mode, group_size=self.gs))

    def run(self, F, **more):
        a, kw = self.args()
        return F.paged_tree_attention(*a, **kw, **more)

    def ref(self):
        values = chunk_values([x.cpu() for x in self.cache], self.fmt, self.mode, self.gs)
        return tree_ref(self.q.cpu(), self.offsets, self.parents, self.lens, self.bt, values,
                        self.hkv, self.sm, self.bs, self.fmt, self.mode, self.window, self.prefix,
                        self.cap, self.slopes,
                        self.cache[2].cpu() if self.mode == STATIC else None, device=DEV)

    def check(self, F, what=""):
        ref = self.ref()
        worst = 0.0
        for dt in (torch.float32, torch.bfloat16):
            out = self.run(F, out_dtype=dt)
            assert F.get_device_error() == 0
            worst = max(worst, check_tree(out, ref, self.d, dt == torch.bfloat16, self.cap,
                                          f"{what} {dt}"))
        return worst


# context lengths ahead of the trees, and trees: none, one token, odd ones, one that crosses
# tiles of tokens, some with nothing ahead
CTX = [0, 1, 15, 127, 128, 129, 300, 1000, 0, 77]
NODES = [5, 1, 3, 1, 7, 2, 31, 16, 64, 0]

FORMATS = [(E4M3, TOKEN_HEAD, 32), (E5M2, TOKEN_HEAD, 32), (INT8, TOKEN_HEAD, 32),
           (E4M3, STATIC, 32), (E5M2, STATIC, 32), (INT8, STATIC, 32), (E4M3, SEGMENT, 32),
           (INT8, SEGMENT, 32), (E4M3, MX, 32), (E4M3, MX, 16), (E5M2, MX, 32), (E5M2, MX, 16)]


@pytest.mark.parametrize("fmt,mode,gs", FORMATS)
@pytest.mark.parametrize("d,bs,hq,hkv", [(128, 16, 16, 2), (64, 32, 12, 4), (128, 64, 3, 1)])
def test_formats(F, fmt, mode, gs, d, bs, hq, hkv):
    Case(1, CTX, NODES, hq, hkv, d, bs, fmt, mode, gs).check(F, f"{fmt} {mode}")


@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 1), (5, 1), (8, 1), (24, 3), (16, 1), (64, 8), (33, 1)])
def test_head_counts(F, hq, hkv):
    Case(2, CTX, NODES, hq, hkv, 128, 16, E4M3, TOKEN_HEAD).check(F)
    Case(3, CTX, NODES, hq, hkv, 64, 16, INT8, TOKEN_HEAD).check(F)


@pytest.mark.parametrize("fmt,mode", [(E4M3, TOKEN_HEAD), (E5M2, STATIC), (INT8, TOKEN_HEAD), (E4M3, MX)])
@pytest.mark.parametrize("mods", [
    dict(window=1), dict(window=3), dict(window=40, prefix=[4] * 10), dict(window=200, cap=20.0),
    dict(cap=50.0), dict(cap=100.0), dict(alibi=True), dict(alibi=True, cap=30.0),
    dict(window=129, alibi=True, prefix=[0, 5, 99, 1, 128, 129, 7, 500, 3, 2]),
    dict(prefix=[2 ** 31 - 1] * 5 + [-5] * 5, window=2), dict(window=2 ** 31 - 1),
    dict(cap=300.0, alibi=True, window=64)])
def test_modifiers(F, fmt, mode, mods):
    Case(4, CTX, NODES, 16, 2, 128, 16, fmt, mode, **mods).check(F, str(mods))
    Case(5, CTX, NODES, 8, 4, 64, 64, fmt, mode, **mods).check(F, str(mods))


@pytest.mark.parametrize("nodes", [1, 2, 4, 5, 8, 9, 16, 17, 31, 32, 33, 64, 65, 128, 200, 256])
def test_tree_sizes(F, nodes):
    """Every share of a row tile, and trees of several."""
    for g, fmt in ((8, E4M3), (1, E4M3), (4, INT8)):
        Case(nodes, [500, 130], [nodes, max(1, nodes // 3)], 2 * g, 2, 128, 16, fmt, TOKEN_HEAD,
             kinds=["any", "roots"]).check(F, f"{nodes} x {g}")


@pytest.mark.parametrize("fmt,mode", [(E4M3, TOKEN_HEAD), (INT8, TOKEN_HEAD), (E5M2, MX)])
def test_long_contexts_split_over_the_gpu(F, fmt, mode):
    Case(6, [20000, 3], [6, 4], 8, 1, 128, 16, fmt, mode).check(F)
    Case(7, [9000, 4500, 12000], [40, 9, 1], 16, 2, 128, 32, fmt, mode, alibi=True).check(F)
    Case(8, [30000], [17], 4, 2, 64, 64, fmt, mode, window=5000, prefix=[200]).check(F)


def test_many_small_requests(F):
    rng = np.random.default_rng(9)
    n = 700
    Case(9, rng.integers(0, 90, n), rng.integers(0, 9, n), 4, 2, 64, 16, E4M3, TOKEN_HEAD).check(F)


def test_negative_and_large_scales_of_scores(F):
    for sm in (-0.1, 3.0, 1e-4):
        Case(10, CTX, NODES, 16, 2, 128, 16, E4M3, TOKEN_HEAD, sm=sm).check(F, str(sm))


def test_rows_of_zeros_and_of_extremes(F):
    c = Case(11, CTX, NODES, 16, 2, 128, 16, E4M3, TOKEN_HEAD)
    c.q[::3] = 0
    c.q[1::3] *= 2.0 ** 40
    c.q[2::3, :, 5] *= 2.0 ** 20
    c.sm = 2.0 ** -45
    c.check(F)
    c.q[1::3] *= 2.0 ** -100
    c.sm = 1.0
    c.check(F)


def test_a_line_is_a_causal_chunk_and_a_node_a_decode(F):
    c = Case(12, [700, 45, 3000], [20, 9, 1], 16, 2, 128, 16, E4M3, TOKEN_HEAD, kinds=["line"])
    a, kw = c.args()
    want = F.paged_prefill_attention(a[0], a[1], *a[3:], **kw, out_dtype=torch.float32)
    ref = c.ref()
    got = c.run(F, out_dtype=torch.float32)
    check_tree(got, ref, 128)
    assert (got - want).abs().max() <= 2.0 ** -9 * want.abs().max()


def test_every_pool_page_order_and_addresses_past_4_gib(F):
    """Blocks of a pool of 300,000 pages of 16 KB each."""
    nb, hkv, bs, d = 300000, 8, 16, 128
    c = Case(13, [400, 129], [7, 20], 16, 8, d, bs, E4M3, TOKEN_HEAD)
    small = c.bt.numpy()
    used = np.unique(small[small >= 0])
    far = np.full(int(small.max()) + 1, -1, np.int64)
    far[used] = np.sort(np.random.default_rng(1).permutation(nb - 270000)[:len(used)]) + 270000
    kc, vc, ks, vs = (torch.zeros((nb,) + tuple(x.shape[1:]), dtype=x.dtype, device=DEV)
                      for x in c.cache)
    for big, x in zip((kc, vc, ks, vs), c.cache):
        big[torch.from_numpy(far[used]).to(DEV)] = x[torch.from_numpy(used).to(DEV)]
    ref = c.ref()
    c.cache = [kc, vc, ks, vs]
    c.bt = torch.from_numpy(np.where(small >= 0, far[np.maximum(small, 0)], -1).astype(np.int32))
    got = c.run(F, out_dtype=torch.float32)
    assert F.get_device_error() == 0
    check_tree(got, ref, d)


# ------------------------------------------------------------------ what is masked does not count
@pytest.mark.parametrize("fmt,mode", [(E4M3, TOKEN_HEAD), (E5M2, TOKEN_HEAD), (E5M2, STATIC),
                                      (E4M3, SEGMENT), (E4M3, MX)])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(F, fmt, mode):
    """A drafted token whose V (or scale) is not finite: only it and its descendants see it;
    what lies behind the last token, and what the window leaves, no row does."""
    nan = 0x7F if fmt == E4M3 else 0x7D
    for window in (0, 100):
        c = Case(14, [140, 300], [12, 9], 8, 2, 128, 16, fmt, mode, window=window,
                 kinds=["any", "roots"])
        ref = c.ref()
        kc, vc, ks, vs = c.cache
        sick = 5  # a node of the first tree
        from tree_ref import lines
        sees = np.array([sick in x for x in lines(c.parents[:12])])

        def row(b, j):
            return int(c.bt[b, j // 16]), j % 16

        p, o = row(0, 140 + sick)
        vc[p, :, o, 3] = nan
        for b in range(2):  # behind the request's end: the rest of its last page
            p, o = row(b, int(c.lens[b]) - 1)
            kc[p, :, o + 1:], vc[p, :, o + 1:] = nan, nan
            if mode == TOKEN_HEAD:
                ks[p, :, o + 1:], vs[p, :, o + 1:] = float("nan"), float("inf")
            if mode == MX:
                ks[p, :, o + 1:], vs[p, :, o + 1:] = 255, 255
        if window:  # outside of every row's window
            p, o = row(1, 300 - window - 3)
            kc[p, :, o], vc[p, :, o] = nan, nan
        out = c.run(F, out_dtype=torch.float32)
        assert F.get_device_error() == 0
        bad = (~torch.isfinite(out)).any(-1).any(-1).cpu().numpy()
        want = np.concatenate([sees, np.zeros(9, bool)])
        assert np.array_equal(bad, want)
        assert (~torch.isfinite(out)).any(-1).all(-1).cpu().numpy()[want].all()
        keep = ~want
        check_tree(out[torch.from_numpy(keep).to(DEV)], tuple(x[keep] if isinstance(x, np.ndarray)
                                                              else x for x in ref), 128)


def test_a_scale_that_is_not_finite_reaches_the_rows_that_see_it(F):
    for what in (2, 3):
        for x in (float("inf"), float("nan")):
            c = Case(15, [256, 40], [6, 3], 8, 2, 128, 16, E4M3, TOKEN_HEAD)
            c.cache[what][int(c.bt[0, 3]), 1, 4] = x  # a context token of request 0, KV head 1
            out = c.run(F, out_dtype=torch.float32)
            bad = (~torch.isfinite(out)).any(-1).cpu().numpy()
            want = np.zeros((9, 8), bool)
            want[:6, 4:] = True
            if what == 3 or x != x:
                assert np.array_equal(bad, want)
            else:  # infinite scores of either sign
                assert not bad[~want].any()


# ------------------------------------------------------------------ bad arguments on the device
def test_bad_parents_count_as_roots(F):
    c = Case(16, [60, 60], [6, 6], 8, 2, 128, 16, E4M3, TOKEN_HEAD)
    c.parents[:] = [-1, 1, 0, -2, 2 ** 31 - 1, 4, -1, 0, 1, 2, 3, -2 ** 31]
    out = c.run(F, out_dtype=torch.float32)
    assert F.get_device_error() == 64
    check_tree(out, c.ref(), 128)  # the reference's lines take them as roots


def test_requests_that_are_skipped_leave_their_rows(F):
    ctx, nodes = [50, 60, 70, 80, 90], [4, 257, 5, 6, 7]
    c = Case(17, ctx, nodes, 8, 2, 128, 16, E4M3, TOKEN_HEAD)
    ref = c.ref()
    for change, flag, gone in (
            (lambda: None, 64, [1]),
            (lambda: c.lens.__setitem__(2, 4), 64 | 4, [1, 2]),
            (lambda: c.lens.__setitem__(3, -1), 64 | 4, [1, 2, 3]),
            (lambda: c.lens.__setitem__(0, 10 ** 6), 64 | 4, [0, 1, 2, 3])):
        change()
        out = torch.full((int(c.offsets[-1]), 8, 128), 7.0, device=DEV)
        c.run(F, out=out)
        assert F.get_device_error() == flag
        rows = np.concatenate([np.full(n, i) for i, n in enumerate(nodes)])
        left = np.isin(rows, gone)
        assert (out.cpu().numpy()[left] == 7.0).all()
        check_tree(out[torch.from_numpy(~left).to(DEV)], tuple(x[~left] for x in ref), 128)


def test_bad_offsets_skip_their_request(F):
    c = Case(18, [50, 60, 70], [4, 5, 6], 8, 2, 128, 16, E4M3, TOKEN_HEAD)
    ref = c.ref()
    # the rows that stay one request's (with offsets 0 4 3 15 row 3 is two requests': either's)
    for off, rows in (([0, 4, 9, 16], range(0, 9)), ([0, 4, 3, 15], range(0, 3)),
                      ([-1, 4, 9, 15], range(4, 15))):
        good = c.offsets.copy()
        c.offsets[:] = off
        out = torch.full((15, 8, 128), 7.0, device=DEV)
        c.run(F, out=out)
        # (the overlapping request's parents are those of other trees: out of order, too)
        assert F.get_device_error() & ~64 == 32
        rows = list(rows)
        check_tree(out[rows], tuple(x[rows] for x in ref), 128)
        if off[0] < 0:
            assert (out[:4] == 7.0).all()
        c.offsets[:] = good


def test_bad_blocks_are_masked(F):
    c = Case(19, [200, 90], [8, 5], 8, 2, 128, 16, E4M3, TOKEN_HEAD)
    ref = None
    bt = c.bt.clone()
    c.bt[0, 3], c.bt[1, 1] = -1, 10 ** 6
    out = c.run(F, out_dtype=torch.float32)
    assert F.get_device_error() == 2
    # the same with those tokens' scores far below: their K^ scaled away is not a mask, so the
    # reference drops the pages
    keep = [[i for i in range(bt.shape[1]) if (b, i) not in ((0, 3), (1, 1))] for b in range(2)]
    lens = c.lens - 16
    tables = torch.stack([torch.cat([bt[b, keep[b]], torch.tensor([-1], dtype=torch.int32)])
                          for b in range(2)])
    c.bt, c.lens = tables, lens
    ref = c.ref()
    check_tree(out, ref, 128)


def test_rows_outside_every_tree_and_empty_batches(F):
    c = Case(20, [50, 60], [4, 5], 8, 2, 128, 16, E4M3, TOKEN_HEAD)
    ref = c.ref()
    c.q = torch.cat([c.q[:4], torch.full((3, 8, 128), float("nan"), device=DEV).bfloat16(), c.q[4:]])
    c.parents = np.concatenate([c.parents[:4], [99, 99, 99], c.parents[4:]]).astype(np.int32)
    a, kw = c.args()
    lens2 = torch.cat([a[8][:1], torch.zeros(1, dtype=torch.int32, device=DEV), a[8][1:]])
    bt2 = torch.cat([a[7][:1], torch.full_like(a[7][:1], -1), a[7][1:]])
    # a request of no nodes between the two, whose offsets step over three rows
    off = torch.tensor([0, 4, 4, 12], dtype=torch.int32, device=DEV)
    out = torch.full((12, 8, 128), 7.0, device=DEV)
    off[2] = 7
    args = (c.q, off, a[2], *a[3:7], bt2, lens2, a[9], a[10])
    F.paged_tree_attention(*args, **kw, out=out)
    assert F.get_device_error() == 4  # the one between is shorter than its three rows
    assert (out[4:7] == 7.0).all()
    check_tree(torch.cat([out[:4], out[7:]]), ref, 128)
    empty = F.paged_tree_attention(c.q[:0], off[:1], a[2][:0], *a[3:7], bt2[:0], lens2[:0], a[9], a[10])
    assert tuple(empty.shape) == (0, 8, 128)


# ------------------------------------------------------------------ streams and graphs
def test_captured_replayed_and_on_another_stream(F):
    c = Case(21, [800, 90, 300], [9, 14, 1], 16, 2, 128, 16, E4M3, TOKEN_HEAD)
    a, kw = c.args()
    want = F.paged_tree_attention(*a, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = F.paged_tree_attention(*a, **kw, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = F.paged_tree_attention(*a, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    q = a[0].clone()
    a[0].copy_(torch.randn_like(q.float()).bfloat16())
    want = F.paged_tree_attention(*a, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert F.get_device_error() == 0


def test_a_larger_batchs_workspace_serves_a_smaller_one(F):
    c = Case(22, [800, 90, 300], [9, 14, 1], 16, 2, 128, 16, E4M3, TOKEN_HEAD)
    want = c.run(F)
    ws = torch.empty(F.tree_workspace_bytes(500, 40, 16, 2, 128, 16, 9999), dtype=torch.uint8, device=DEV)
    ws.random_(0, 256)
    assert torch.equal(c.run(F, workspace=ws), want)


@pytest.mark.parametrize("fmt,mode,d", [(INT8, TOKEN_HEAD, 128), (E4M3, MX, 64), (E5M2, STATIC, 128)])
def test_row_blocks_of_every_kind_in_one_range(F, fmt, mode, d):
    """Shared lanes, blocks of up to 128 and of 256 rows behind one another on an SM, and the
    same call again."""
    rng = np.random.default_rng(23)
    nodes = [int(n) for n in rng.choice([0, 1, 4, 9, 16, 17, 32, 33, 64, 100], 60)]
    ctx = [int(c) for c in rng.integers(0, 900, 60)]
    c = Case(23, ctx, nodes, 32, 4, d, 16, fmt, mode)
    c.check(F)
    want = c.run(F)
    for _ in range(10):
        assert torch.equal(c.run(F), want)
