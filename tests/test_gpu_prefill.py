"""Attention of ragged query chunks against the 64-bit reference."""
import numpy as np
import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def F():
    import fp8_quantised_paged_gb300 as F
    torch.cuda.set_device(0)
    F.get_device_error()
    return F


class Batch:
    """Requests of `lens` cached tokens whose last `chunks` are queries."""

    def __init__(self, lens, chunks, hq, hkv, d, bs, fmt, mode, gs=32, seed=0, qgain=1.0,
                 reach=0):
        rng = np.random.default_rng(seed)
        self.bt, nb = R.make_tables(rng, lens, bs)
        more = reach // bs - self.bt.shape[1]
        if more > 0:
            self.bt = torch.cat([self.bt, torch.full((len(lens), more), -1, dtype=torch.int32)], 1)
        self.cache = list(R.make_cache(rng, nb, hkv, bs, d, fmt, mode, gs))
        self.lens, self.chunks = list(lens), list(chunks)
        self.offsets = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
        n = int(self.offsets[-1])
        self.q = torch.from_numpy(rng.standard_normal((n, hq, d)) * qgain).bfloat16()
        self.hq, self.hkv, self.d, self.bs = hq, hkv, d, bs
        self.form = dict(fmt=fmt, scale_mode=mode, group_size=gs)
        self.sm = d ** -0.5

    def values(self):
        f = self.form
        return R.chunk_values(self.cache, f["fmt"], f["scale_mode"], f["group_size"])

    def ref(self, device="cpu", **mods):
        return R.chunk_ref(self.q, self.offsets, self.lens, self.bt, self.values(), self.hkv,
                           self.sm, self.bs, device=device, **mods)

    def args(self):
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
        return (self.q.to(DEV), i32(self.offsets), *(t.to(DEV) for t in self.cache),
                self.bt.to(DEV), i32(self.lens), self.hkv, self.sm)

    def run(self, F, window=0, prefix=None, cap=0.0, slopes=None, out_dtype=torch.float32, **kw):
        return F.paged_prefill_attention(
            *self.args(), window=window,
            prefix_lens=None if prefix is None else torch.tensor(prefix, dtype=torch.int32,
                                                                 device=DEV),
            logit_cap=cap, alibi_slopes=None if slopes is None else slopes.to(DEV),
            out_dtype=out_dtype, **self.form, **kw)

    def check(self, F, what="", **mods):
        ref = self.ref(**mods)
        for dt in (torch.float32, torch.bfloat16):
            got = self.run(F, out_dtype=dt, **mods)
            R.check(got, ref, self.d, bf16=dt == torch.bfloat16,
                    half=self.form["scale_mode"], cap=mods.get("cap", 0.0), what=f"{what} {dt}")
        assert F.get_device_error() == 0
        return got


def slopes_of(hq):
    return torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).float()


LENS = [1, 5, 17, 64, 130, 200, 257, 390]
CHUNKS = [1, 5, 3, 64, 1, 150, 129, 16]
KINDS = [(R.E4M3, R.TOKEN_HEAD, 32), (R.E5M2, R.STATIC, 32), (R.INT8, R.TOKEN_HEAD, 32),
         (R.E4M3, R.MX, 32), (R.E5M2, R.MX, 16), (R.E4M3, R.SEGMENT, 32), (R.INT8, R.STATIC, 32),
         (R.E5M2, R.TOKEN_HEAD, 32), (R.INT8, R.SEGMENT, 32)]


@pytest.mark.parametrize("fmt,mode,gs", KINDS)
@pytest.mark.parametrize("d,hq,hkv,bs", [(128, 8, 2, 16), (64, 4, 1, 32), (128, 6, 2, 64)])
def test_formats_and_scale_modes(F, fmt, mode, gs, d, hq, hkv, bs):
    Batch(LENS, CHUNKS, hq, hkv, d, bs, fmt, mode, gs).check(F)


@pytest.mark.parametrize("fmt,mode,gs", KINDS)
@pytest.mark.parametrize("d", [64, 128])
def test_all_modifiers_together(F, fmt, mode, gs, d):
    b = Batch(LENS, CHUNKS, 8, 2, d, 16, fmt, mode, gs, seed=1)
    b.check(F, window=40, prefix=[3, 0, 5, 100, 17, 190, 1, 64], cap=3.0, slopes=slopes_of(8))


# Heads per KV head that make the chunks below long: rows are queries times heads,
# and from 768 rows a request on, tiles are converted once for all row blocks, if
# the tables have room for more than 256 tokens (REACH).
LONG, REACH = 96, 320


@pytest.mark.parametrize("fmt,mode,gs", KINDS)
@pytest.mark.parametrize("d,hkv,bs", [(128, 1, 16), (64, 2, 64)])
@pytest.mark.parametrize("mods", [{}, {"window": 40, "prefix": [3, 0, 150, 300, 1], "cap": 3.0}])
def test_long_chunks_of_every_format(F, fmt, mode, gs, d, hkv, bs, mods):
    b = Batch([130, 17, 200, 390, 1], [1, 17, 64, 50, 1], LONG * hkv, hkv, d, bs, fmt, mode, gs,
              seed=19)
    if mods:
        mods = dict(mods, slopes=slopes_of(LONG * hkv))
    ref = b.ref(device=DEV, **mods)
    got = b.run(F, **mods)
    R.check(got, ref, d, half=mode, cap=mods.get("cap", 0.0))
    assert F.get_device_error() == 0


@pytest.mark.parametrize("window", [0, 1, 2, 16, 17, 100, 128, 257, 5000])
@pytest.mark.parametrize("prefix", [None, 0, 1, 40, 150, 400, -3])
def test_windows_and_prefixes(F, window, prefix):
    b = Batch(LENS, CHUNKS, 8, 1, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=2)
    b.check(F, window=window, prefix=None if prefix is None else [prefix] * len(LENS))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 5), (7, 1), (16, 1), (32, 2), (129, 1),
                                    (300, 1)])
def test_head_groups_of_any_size(F, hq, hkv):
    Batch([70, 3, 131], [33, 3, 2], hq, hkv, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=3).check(F)


@pytest.mark.parametrize("cap", [0.01, 1.0, 30.0, 1e4, 1e30])
@pytest.mark.parametrize("gain", [0.1, 30.0])
def test_caps_far_below_and_far_above_the_scores(F, cap, gain):
    Batch([77, 5, 300], [20, 5, 9], 4, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=5,
          qgain=gain).check(F, cap=cap)


def test_distance_bias_at_steep_and_flat_slopes(F):
    sl = torch.tensor([0.0, 1e-4, 0.01, 0.5, 4.0, 100.0, -0.02, 1.0])
    Batch([900, 1, 33], [60, 1, 33], 8, 1, 128, 16, R.E5M2, R.TOKEN_HEAD, seed=6).check(
        F, slopes=sl)
    Batch([300, 33], [60, 33], 8, 1, 128, 16, R.E5M2, R.TOKEN_HEAD, seed=6).check(
        F, slopes=sl, prefix=[290, 20])


@pytest.mark.parametrize("kw", [{}, {"window": 700}, {"prefix": [900, 5]}, {"cap": 20.0}])
def test_long_contexts(F, kw):
    b = Batch([4100, 1337], [300, 1337], 8, 1, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=7)
    ref = b.ref(device=DEV, **kw)
    cap = kw.get("cap", 0.0)
    R.check(b.run(F, **kw), ref, 128, half=R.TOKEN_HEAD, cap=cap)
    R.check(b.run(F, out_dtype=torch.bfloat16, **kw), ref, 128, bf16=True, half=R.TOKEN_HEAD, cap=cap)


@pytest.mark.parametrize("n,count", [(300, 12), (200, 16), (40, 60), (70, 30)])
@pytest.mark.parametrize("kw", [{}, {"cap": 20.0}])
def test_many_short_items_whose_last_block_has_one_row_tile(F, n, count, kw):
    """A row block of at most 128 rows leaves the second row tile idle, whose threads
    run ahead to their next block: what they read there has to be that block's.
    300 queries: 2400 rows, ten row blocks, tiles converted once; the others by each."""
    b = Batch([n] * count, [n] * count, 64, 8, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=20)
    ref = b.ref(device=DEV, **kw)
    outs = [b.run(F, **kw) for _ in range(6)]
    for got in outs:
        R.check(got, ref, 128, half=R.TOKEN_HEAD, cap=kw.get("cap", 0.0))
        assert torch.equal(got, outs[0])
    assert F.get_device_error() == 0


@pytest.mark.parametrize("hq", [4, 2 * 452])
def test_requests_without_queries_or_tokens(F, hq):
    b = Batch([40, 0, 17, 9, 0], [0, 0, 17, 0, 0], hq, 2, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=8,
              reach=REACH)
    b.check(F)


def test_rows_outside_the_chunks_are_left_alone(F):
    b = Batch([40, 30], [40, 7], 4, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=9)
    ref = b.ref()
    pad = torch.randn(9, 4, 128).bfloat16()
    b.q = torch.cat([pad[:4], b.q, pad[4:]])
    b.offsets = b.offsets + 4
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((56, 4, 128), 77.0, dtype=dt, device=DEV)
        assert b.run(F, out=out, out_dtype=dt) is out
        assert (out[:4] == 77).all() and (out[51:] == 77).all()
        R.check(out[4:51], ref, 128, bf16=dt == torch.bfloat16, half=R.TOKEN_HEAD)


@pytest.mark.parametrize("fmt,nan", [(R.E4M3, 0x7F), (R.E5M2, 0x7E), (R.E5M2, 0x7C)])
@pytest.mark.parametrize("bad_scale", [float("nan"), float("inf"), 1.0])
@pytest.mark.parametrize("hq", [8, LONG * 2])
def test_what_masked_tokens_hold_does_not_matter(F, fmt, nan, bad_scale, hq):
    """Past the end of the request, before the window and, for all but the last
    query, after it: what a row does not see may be anything."""
    lens, chunks = [70, 50, 33, 17], [9, 50, 1, 4]
    b = Batch(lens, chunks, hq, 2, 128, 16, fmt, R.TOKEN_HEAD, seed=10, reach=REACH)
    mods = dict(window=20, prefix=[5, 0, 2, 0])
    ref = b.ref(**mods)
    kc, vc, ks, vs = b.cache
    last = []
    for r, L in enumerate(lens):
        first = L - chunks[r] - 20 + 1  # the first query's window
        last.append(int(b.offsets[r + 1]) - 1)
        for j in range(b.bt.shape[1] * 16):
            blk = int(b.bt[r, j // 16])
            # unseen by all, or the last token: seen by the last query alone
            if blk < 0 or not (j >= L - 1 or (j < first and j >= mods["prefix"][r])):
                continue
            for c, sc in ((kc, ks), (vc, vs)):
                c[blk, :, j % 16] = nan
                sc[blk, :, j % 16] = bad_scale
    got = b.run(F, **mods)
    keep = [i for i in range(int(b.offsets[-1])) if i not in last]
    R.check(got[keep], tuple(x[keep] for x in ref), 128, half=R.TOKEN_HEAD)


@pytest.mark.parametrize("fmt,mode", [(R.E4M3, R.TOKEN_HEAD), (R.INT8, R.TOKEN_HEAD),
                                      (R.E4M3, R.MX)])
def test_a_huge_scale_beside_small_ones(F, fmt, mode):
    """Tokens whose scales are 2^22 times their neighbours', in every group of 32: rows
    that mask them keep their precision.

    The bound, with S the largest scale (a request's largest small one, top, times
    2^22) and rho the smallest over the largest of a group: K^ and V^ are held in units
    that put S between 2^6 and 2^7, and a scale is split into two f16 halves, off by at
    most 2^-25: 2^-31 / rho relative to the token (MX scales: exact).  A product below
    the normal range is off by 2^-25 more: 2^-31 S in V^, and sm sum |q| 2^-31 S in a
    score.  The term of P is 2^-36 S sum |code|, as ever."""
    up, win = 22, 4
    b = Batch([90, 40], [60, 33], 4, 2, 128, 16, fmt, mode, seed=17, qgain=0.01)
    out, A, Z, B, W, Fl = b.ref(window=win)
    *_, vscale, kscale = b.values()
    top = float(max(vscale.max(), kscale.max()))
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
    rel = 0.0 if mode == R.MX else 2.0 ** -31 / rho
    for r in range(2):  # W without its own floor, 2^-24 of the request's largest scale
        own = vscale[b.bt[r, :(b.lens[r] + 15) // 16].long()].transpose(0, 1).flatten(1, 2)
        own = own[:, :b.lens[r]].amax((1, 2)).repeat_interleave(2).numpy()[:, None]
        W[b.offsets[r]:b.offsets[r + 1]] -= 2.0 ** -24 * own
    W = 2.0 ** up * (W + 2.0 ** -31 * top) + rel * A
    Fl = 2.0 ** (up - 7) * Fl + rel * Z
    got = b.run(F, window=win)
    keep = []
    for r in range(2):
        for i in range(b.chunks[r]):
            pos = b.lens[r] - b.chunks[r] + i
            if not any(pos - win < j <= pos for j in huge):
                keep.append(int(b.offsets[r]) + i)
    R.check(got[keep], tuple(x[keep] for x in (out, A, Z, B, W, Fl)), 128, half=mode)
    assert F.get_device_error() == 0


@pytest.mark.parametrize("sm", [0.0, -0.1, 1e-30])
@pytest.mark.parametrize("cap", [0.0, 5.0])
def test_scale_factors_of_zero_and_below(F, sm, cap):
    b = Batch([70, 20], [30, 20], 4, 2, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=18)
    b.sm = sm
    b.check(F, window=9, cap=cap, slopes=slopes_of(4))


@pytest.mark.parametrize("hq", [4, LONG])
def test_pages_no_query_sees_are_not_read(F, hq):
    b = Batch([400, 200], [30, 8], hq, 1, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=11)
    mods = dict(window=33, prefix=[18, 0])
    ref = b.ref(**mods)
    b.bt[0, 2:(400 - 30 - 33) // 16] = -1
    b.bt[1, :(200 - 8 - 33) // 16] = 10 ** 6
    R.check(b.run(F, **mods), ref, 64, half=R.TOKEN_HEAD)
    assert F.get_device_error() == 0


@pytest.mark.parametrize("hq", [4, 1536])
def test_bad_blocks_lengths_and_offsets_are_flagged(F, hq):
    from fp8_quantised_paged_gb300 import _native as N
    b = Batch([40, 20, 10], [5, 2, 3], hq, 1, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=12,
              reach=REACH)
    b.bt[0, 1] = 10 ** 6
    b.lens[1], b.lens[2] = 10 ** 7, -4
    got = b.run(F)
    assert torch.isfinite(got[:5]).all() and not got[7:].any()
    assert F.get_device_error() == N.DEVERR_BLOCK_RANGE | N.DEVERR_SEQ_LEN
    # a chunk longer than its request: the rows before position 0 see nothing
    b = Batch([4, 20], [4, 2], hq, 1, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=12,
              reach=REACH)
    ref = b.ref()
    b.lens[0] = 2
    got = b.run(F)
    assert not got[:2].any() and got[2:].any()
    R.check(got[4:], tuple(x[4:] for x in ref), 64, half=R.TOKEN_HEAD)
    assert F.get_device_error() == N.DEVERR_SEQ_LEN
    for bad in ([0, 9, 6], [-1, 4, 6], [0, 4, 7]):
        b = Batch([4, 20], [4, 2], hq, 1, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=12,
              reach=REACH)
        b.offsets = np.array(bad, np.int32)
        out = torch.full((6, hq, 64), 7.0, device=DEV)
        b.run(F, out=out)
        assert F.get_device_error() & N.DEVERR_Q_OFFSETS


@pytest.mark.parametrize("hq", [8, 48])
def test_graphs_that_share_a_workspace_and_other_streams(F, hq):
    b = Batch([300, 7, 64], [200, 7, 1], hq, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=13)
    ws = torch.empty(F.prefill_workspace_bytes(208, 3, hq, 2, 128, 16, b.bt.shape[1]),
                     dtype=torch.uint8, device=DEV)
    args = b.args()
    kws = [dict(window=50), dict(logit_cap=5.0)]
    run = lambda kw, **o: F.paged_prefill_attention(*args, **b.form, **kw, **o)  # noqa: E731
    want = [run(kw, workspace=ws).clone() for kw in kws]
    outs, graphs = [torch.zeros_like(w) for w in want], []
    for kw, o in zip(kws, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(kw, out=o, workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(kws[0], stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])


def test_calls_at_once_on_several_streams(F):
    """Both head sizes, both ways of conversion and a decode, each on a stream of its
    own and all under way together."""
    form = dict(fmt=R.E4M3, mode=R.TOKEN_HEAD)
    batches = [Batch([900, 40], [300, 40], 8, 2, 128, 16, *form.values(), seed=21),
               Batch([700] * 3, [9] * 3, 8, 2, 64, 16, *form.values(), seed=22),
               Batch([1500], [700], 16, 4, 64, 32, *form.values(), seed=23),
               Batch([2000] * 4, [5] * 4, 8, 2, 128, 64, *form.values(), seed=24)]
    args = [b.args() for b in batches]
    calls = [lambda a=a, b=b, **kw: F.paged_prefill_attention(*a, **b.form, **kw)
             for a, b in zip(args, batches)]
    dec = Batch([3000, 17], [1, 1], 8, 2, 128, 16, *form.values(), seed=25)
    q, _, *rest = dec.args()
    calls.append(lambda **kw: F.paged_decode_attention_mod(q, *rest, **dec.form, window=700, **kw))
    want = [c().clone() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    outs = [[] for _ in calls]
    for _ in range(15):
        for c, st, o in zip(calls, streams, outs):
            o.append(c(stream=st))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, w) for x in o)
    assert F.get_device_error() == 0


def test_repeated_calls_are_bit_identical(F):
    b = Batch([3000, 40, 1777], [500, 40, 33], 8, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=14)
    outs = [b.run(F, window=900, cap=20.0) for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_offsets_past_32_bits(F):
    hkv, bs, d, fmt = 8, 64, 128, R.E4M3
    nb = (1 << 32) // (hkv * bs * d) + 40
    b = Batch([150], [40], hkv, hkv, d, bs, fmt, R.TOKEN_HEAD, seed=15)
    ref = b.ref()
    args = list(b.args())
    for i, t in zip(range(2, 6), list(args[2:6])):
        w = torch.empty((nb,) + tuple(t.shape[1:]), dtype=t.dtype, device=DEV)
        w[nb - t.shape[0]:] = t
        args[i] = w
    args[6] = torch.where(args[6] >= 0, args[6] + nb - b.cache[0].shape[0], -1).int()
    got = F.paged_prefill_attention(*args, out_dtype=torch.float32, **b.form)
    R.check(got, ref, d, half=R.TOKEN_HEAD)


def test_the_operators_in_a_row(F):
    """A server's use: prompts appended with rotation and prefilled in two chunks,
    then decode steps, under a window with kept first tokens and capped scores;
    each attention against the reference on the cache as it stands."""
    hq, hkv, d, bs, fmt = 8, 2, 128, 16, R.E4M3
    rng = np.random.default_rng(16)
    plen, steps = [150, 33, 1], 3
    bt, nb = R.make_tables(rng, [n + steps for n in plen], bs)
    g = torch.Generator().manual_seed(16)
    half = d // 2
    ang = torch.arange(400, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(half, dtype=torch.float64) / half)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    kc = torch.zeros(nb, hkv, bs, d, dtype=torch.uint8, device=DEV)
    vc, ks = torch.zeros_like(kc), torch.zeros(nb, hkv, bs, 1, device=DEV)
    vs = torch.zeros_like(ks)
    form = dict(fmt=fmt, scale_mode=R.TOKEN_HEAD)
    mods = dict(window=60, cap=8.0)
    prefix = torch.tensor([4, 4, 4], dtype=torch.int32)
    lens = [0, 0, 0]

    def step(counts, decode):
        n = sum(counts)
        qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g).bfloat16().to(DEV)
        pos = np.concatenate([np.arange(L, L + c) for L, c in zip(lens, counts)])
        req = np.repeat(np.arange(3), counts)
        slots = np.array([int(bt[r, p // bs]) * bs + p % bs for r, p in zip(req, pos)])
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
        q = F.kv_append_rope(qkv[:, :hq * d].unflatten(1, (hq, d)),
                             qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                             qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)), i32(pos), cs.to(DEV),
                             i32(slots), kc, vc, ks, vs, **form)
        for r in range(3):
            lens[r] += counts[r]
        off = np.concatenate([[0], np.cumsum(counts)])
        common = dict(window=60, prefix_lens=prefix.to(DEV), logit_cap=8.0,
                      out_dtype=torch.float32, **form)
        if decode:
            got = F.paged_decode_attention_mod(q, kc, vc, ks, vs, bt.to(DEV), i32(lens), hkv,
                                               d ** -0.5, **common)
        else:
            got = F.paged_prefill_attention(q, i32(off), kc, vc, ks, vs, bt.to(DEV), i32(lens),
                                            hkv, d ** -0.5, **common)
        values = tuple(x.cpu() for x in R.chunk_values((kc, vc, ks, vs), fmt, R.TOKEN_HEAD, 0))
        ref = R.chunk_ref(q.cpu(), off, lens, bt, values, hkv, d ** -0.5, bs, prefix=prefix,
                          **mods)
        R.check(got, ref, d, half=None if decode else R.TOKEN_HEAD, cap=mods["cap"])
        # the queries and the newest keys really are turned
        want = R.rotate(qkv[:, :hq * d].cpu().unflatten(1, (hq, d)), cs[pos][:, :half],
                        cs[pos][:, half:]).bfloat16()
        assert torch.equal(q.cpu(), want)

    step([100, 20, 1], decode=False)
    step([50, 13, 0], decode=False)
    for _ in range(steps):
        step([1, 1, 1], decode=True)
    assert F.get_device_error() == 0
