"""Decode with score modifiers against the 64-bit reference."""
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
    F.set_decode_workers(0)
    F.get_device_error()
    return F


def setup(lens, hq, hkv, d, bs, fmt, mode, gs=32, seed=0, qgain=1.0):
    rng = np.random.default_rng(seed)
    bt, nb = R.make_tables(rng, lens, bs)
    kc, vc, ks, vs = R.make_cache(rng, nb, hkv, bs, d, fmt, mode, gs)
    q = torch.from_numpy(rng.standard_normal((len(lens), hq, d)) * qgain).bfloat16()
    return q, kc, vc, ks, vs, bt, torch.tensor(lens, dtype=torch.int32)


def call(F, s, hkv, sm, fmt, mode, gs=32, window=0, prefix=None, cap=0.0, slopes=None,
         out_dtype=torch.float32, **kw):
    q, kc, vc, ks, vs, bt, lens = (t.to(DEV) for t in s)
    return F.paged_decode_attention_mod(
        q, kc, vc, ks, vs, bt, lens, hkv, sm, window=window,
        prefix_lens=None if prefix is None else torch.tensor(prefix, dtype=torch.int32,
                                                             device=DEV),
        logit_cap=cap, alibi_slopes=None if slopes is None else slopes.to(DEV), fmt=fmt,
        scale_mode=mode, group_size=gs, out_dtype=out_dtype, **kw)


def reference(s, hkv, sm, fmt, mode, gs=32, **mods):
    q, kc, vc, ks, vs, bt, lens = s
    values = (R.dequant(kc, ks, fmt, mode, gs), R.dequant(vc, vs, fmt, mode, gs))
    return R.attention_ref(q, range(len(lens)), [int(n) - 1 for n in lens], lens, bt, values, hkv,
                           sm, kc.shape[2], **mods)


def both(F, s, hkv, d, sm, fmt, mode, gs=32, **mods):
    ref = reference(s, hkv, sm, fmt, mode, gs, **mods)
    for dt in (torch.float32, torch.bfloat16):
        got = call(F, s, hkv, sm, fmt, mode, gs, out_dtype=dt, **mods)
        R.check(got, ref, d, bf16=dt == torch.bfloat16, cap=mods.get("cap", 0.0), what=f"{dt}")
    assert F.get_device_error() == 0
    return got


def slopes_of(hq):
    return torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).float()


LENS = [0, 1, 2, 15, 16, 17, 31, 64, 65, 200, 333]
KINDS = [(R.E4M3, R.TOKEN_HEAD, 32), (R.E5M2, R.STATIC, 32), (R.INT8, R.TOKEN_HEAD, 32),
         (R.E4M3, R.MX, 32), (R.E5M2, R.MX, 16), (R.E4M3, R.SEGMENT, 32), (R.INT8, R.STATIC, 32)]


@pytest.mark.parametrize("fmt,mode,gs", KINDS)
@pytest.mark.parametrize("d,hq,hkv,bs", [(128, 8, 2, 16), (64, 4, 1, 32), (128, 24, 3, 64)])
def test_all_modifiers_together(F, fmt, mode, gs, d, hq, hkv, bs):
    s = setup(LENS, hq, hkv, d, bs, fmt, mode, gs)
    both(F, s, hkv, d, d ** -0.5, fmt, mode, gs, window=40,
         prefix=[3, 0, 5, 1, 16, 17, 2, 64, 1, 0, 33], cap=3.0, slopes=slopes_of(hq))


@pytest.mark.parametrize("window", [0, 1, 2, 16, 17, 100, 333, 5000])
@pytest.mark.parametrize("prefix", [None, 0, 1, 16, 40, 400, -3])
def test_windows_and_prefixes(F, window, prefix):
    s = setup(LENS, 8, 1, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=3)
    both(F, s, 1, 64, 0.125, R.E4M3, R.TOKEN_HEAD, window=window,
         prefix=None if prefix is None else [prefix] * len(LENS))


@pytest.mark.parametrize("cap", [0.01, 1.0, 30.0, 1e4, 1e30])
@pytest.mark.parametrize("gain", [0.1, 30.0])
def test_caps_far_below_and_far_above_the_scores(F, cap, gain):
    s = setup([77, 5, 300], 4, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=5, qgain=gain)
    both(F, s, 2, 128, 128 ** -0.5, R.E4M3, R.TOKEN_HEAD, cap=cap)


def test_distance_bias_at_steep_and_flat_slopes(F):
    s = setup([900, 1, 33], 8, 1, 128, 16, R.E5M2, R.TOKEN_HEAD, seed=6)
    sl = torch.tensor([0.0, 1e-4, 0.01, 0.5, 4.0, 100.0, -0.02, 1.0])
    both(F, s, 1, 128, 128 ** -0.5, R.E5M2, R.TOKEN_HEAD, slopes=sl)


def test_without_modifiers_it_is_the_plain_decode(F):
    s = setup(LENS, 8, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=7)
    got = call(F, s, 2, 0.09, R.E4M3, R.TOKEN_HEAD)
    q, kc, vc, ks, vs, bt, lens = (t.to(DEV) for t in s)
    want = F.paged_decode_attention(q, kc, vc, ks, vs, bt, lens, 2, 0.09,
                                    out_dtype=torch.float32)
    ref = reference(s, 2, 0.09, R.E4M3, R.TOKEN_HEAD)
    R.check(got, ref, 128)
    R.check(want, ref, 128)


@pytest.mark.parametrize("workers", [1, 2, 3, 7, 50, 1000])
def test_every_split_of_two_page_ranges(F, workers):
    s = setup([0, 700, 40, 1, 512], 8, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=8)
    ref = reference(s, 2, 0.088, R.E4M3, R.TOKEN_HEAD, window=150, prefix=[9, 70, 3, 1, 16])
    try:
        F.set_decode_workers(workers)
        got = call(F, s, 2, 0.088, R.E4M3, R.TOKEN_HEAD, window=150, prefix=[9, 70, 3, 1, 16])
    finally:
        F.set_decode_workers(0)
    R.check(got, ref, 128)


@pytest.mark.parametrize("fmt,nan", [(R.E4M3, 0x7F), (R.E5M2, 0x7E), (R.E5M2, 0x7C)])
@pytest.mark.parametrize("bad_scale", [float("nan"), float("inf"), 1.0])
def test_what_masked_tokens_hold_does_not_matter(F, fmt, nan, bad_scale):
    lens = [70, 50, 33, 17]
    s = setup(lens, 8, 2, 128, 16, fmt, R.TOKEN_HEAD, seed=9)
    mods = dict(window=20, prefix=[5, 0, 2, 0])
    ref = reference(s, 2, 0.088, fmt, R.TOKEN_HEAD, **mods)
    q, kc, vc, ks, vs, bt, _ = s
    for b, L in enumerate(lens):
        for j in range(bt.shape[1] * 16):
            blk = int(bt[b, j // 16])
            if blk < 0 or (j < L and (L - 1 - j < 20 or j < mods["prefix"][b])):
                continue
            for c, sc in ((kc, ks), (vc, vs)):
                c[blk, :, j % 16] = nan
                sc[blk, :, j % 16] = bad_scale
    R.check(call(F, s, 2, 0.088, fmt, R.TOKEN_HEAD, **mods), ref, 128)


def test_pages_outside_the_window_are_not_read(F):
    """The table entries between the prefix and the window may name no block."""
    s = setup([400, 90], 4, 1, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=10)
    mods = dict(window=33, prefix=[18, 0])
    ref = reference(s, 1, 0.125, R.E4M3, R.TOKEN_HEAD, **mods)
    s[5][0, 2:(400 - 33) // 16] = -1
    s[5][1, :(90 - 33) // 16] = 10 ** 6
    R.check(call(F, s, 1, 0.125, R.E4M3, R.TOKEN_HEAD, **mods), ref, 64)
    assert F.get_device_error() == 0


def test_bad_blocks_and_lengths_are_flagged(F):
    from fp8_quantised_paged_gb300 import _native as N
    s = setup([40, 20, 10], 4, 1, 64, 16, R.E4M3, R.TOKEN_HEAD, seed=11)
    s[5][0, 1] = 10 ** 6
    s[6][1] = 10 ** 7
    s[6][2] = -4
    got = call(F, s, 1, 0.125, R.E4M3, R.TOKEN_HEAD, window=30)
    assert torch.isfinite(got[0]).all() and not got[2].any()
    assert F.get_device_error() == N.DEVERR_BLOCK_RANGE | N.DEVERR_SEQ_LEN


@pytest.mark.parametrize("mode", [R.TOKEN_HEAD, R.STATIC])
def test_the_smallest_workspace_that_is_taken_is_not_overrun(F, mode):
    """A workspace below the size function's answer is refused, or used with fewer
    ranges; nothing behind it is written."""
    hq, hkv, d, bs = 64, 8, 128, 32
    s = setup([700, 3, 2000], hq, hkv, d, bs, R.E5M2, mode, seed=14)
    ref = reference(s, hkv, 0.088, R.E5M2, mode, cap=5.0)
    full = F.decode_workspace_bytes(3, hq, hkv, d, d, bs, s[5].shape[1])
    buf = torch.empty(full, dtype=torch.uint8, device=DEV)

    def run(n):
        buf.fill_(0xA5)
        got = call(F, s, hkv, 0.088, R.E5M2, mode, cap=5.0, workspace=buf[:n])
        assert (buf[n:] == 0xA5).all()
        R.check(got, ref, d, cap=5.0)

    low, high = 0, full  # refused, taken
    run(full)
    while high - low > 256:
        n = (low + high) // 512 * 256
        try:
            run(n)
            high = n
        except F.Fp8paError:
            low = n
    run(high)
    assert F.get_device_error() == 0


def test_graphs_that_share_a_workspace_and_other_streams(F):
    hq, hkv, d = 8, 2, 128
    s = setup([300, 7, 64], hq, hkv, d, 16, R.E4M3, R.TOKEN_HEAD, seed=12)
    ws = torch.empty(F.decode_workspace_bytes(3, hq, hkv, d, d, 16, s[5].shape[1]),
                     dtype=torch.uint8, device=DEV)
    dev = [t.to(DEV) for t in s]
    a = dict(window=50, out_dtype=torch.float32, workspace=ws)
    b = dict(logit_cap=5.0, out_dtype=torch.float32, workspace=ws)
    run = lambda kw, **o: F.paged_decode_attention_mod(*dev, hkv, 0.088, **kw, **o)  # noqa: E731
    want = [run(a).clone(), run(b).clone()]
    outs, graphs = [torch.zeros_like(w) for w in want], []
    for kw, o in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(kw, out=o)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(dict(window=50, out_dtype=torch.float32), stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])


def test_repeated_calls_are_bit_identical(F):
    s = setup([3000, 40, 1777], 8, 2, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=13)
    outs = [call(F, s, 2, 0.088, R.E4M3, R.TOKEN_HEAD, window=900, cap=20.0) for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_offsets_past_32_bits(F):
    """A pool of more than 2^32 code bytes: the last blocks hold the request."""
    hkv, bs, d, fmt = 8, 64, 128, R.E4M3
    nb = (1 << 32) // (hkv * bs * d) + 40
    lens = [150]
    rng = np.random.default_rng(14)
    kc, vc, ks, vs = R.make_cache(rng, 3, hkv, bs, d, fmt, R.TOKEN_HEAD)
    q = torch.from_numpy(rng.standard_normal((1, hkv, d))).bfloat16()
    bt = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    s = (q, kc, vc, ks, vs, bt, torch.tensor(lens, dtype=torch.int32))
    ref = reference(s, hkv, 0.088, fmt, R.TOKEN_HEAD, window=100)
    big = []
    for t in (kc, vc, ks, vs):
        w = torch.empty((nb,) + tuple(t.shape[1:]), dtype=t.dtype, device=DEV)
        w[nb - 3:] = t.to(DEV)
        big.append(w)
    got = F.paged_decode_attention_mod(q.to(DEV), *big, (bt + nb - 3).to(DEV), s[6].to(DEV), hkv,
                                       0.088, window=100, out_dtype=torch.float32)
    R.check(got, ref, d)
