"""Refused arguments of the rotary append, the decode with score modifiers and
the prefill: status codes and exceptions, none of which touches a device."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from fp8_quantised_paged_gb300 import build
    build.build()
    from fp8_quantised_paged_gb300 import _native
    return _native.lib


P = ctypes.c_void_p
FAKE = P(0x1000)


def rope(lib, **kw):
    a = dict(q=FAKE, qo=FAKE, k=FAKE, v=FAKE, qs=512, qos=512, ks=128, vs=128, pos=FAKE, cs=FAKE,
             mp=100, rot=64, ro=0, il=0, sl=FAKE, n=4, hq=8, hkv=2, d=64, fmt=0, mode=0, gs=64,
             kc=FAKE, vc=FAKE, ksc=FAKE, vsc=FAKE, nb=8, bs=16)
    a.update(kw)
    return lib.fp8pa_kv_append_rope(
        a["q"], a["qo"], a["k"], a["v"], a["qs"], a["qos"], a["ks"], a["vs"], a["pos"], a["cs"],
        a["mp"], a["rot"], a["ro"], a["il"], a["sl"], a["n"], a["hq"], a["hkv"], a["d"], a["fmt"],
        a["mode"], a["gs"], a["kc"], a["vc"], a["ksc"], a["vsc"], a["nb"], a["bs"], None)


@pytest.mark.parametrize("want,kw", [
    (-1, dict(q=None)), (-1, dict(qo=None)), (-1, dict(k=None)), (-1, dict(pos=None)),
    (-1, dict(cs=None)), (-1, dict(sl=None)), (-1, dict(kc=None)), (-1, dict(vc=None)),
    (-2, dict(fmt=3)), (-2, dict(mode=9)), (-2, dict(il=2)),
    (-3, dict(n=-1)), (-3, dict(hq=0)), (-3, dict(hkv=0)), (-3, dict(d=0)), (-3, dict(mp=0)),
    (-3, dict(rot=0)), (-3, dict(rot=80)), (-3, dict(ro=-8)), (-3, dict(ro=8)),
    (-3, dict(ks=127)), (-3, dict(vs=120)), (-3, dict(qs=504)), (-3, dict(qos=8)),
    (-4, dict(rot=24)), (-4, dict(rot=48, ro=4)), (-4, dict(d=40)), (-4, dict(mode=4)),
    (-4, dict(fmt=2, mode=3, gs=32)), (-4, dict(mode=2, gs=24)),
    (-4, dict(d=576, hkv=1, ks=576, rot=512, q=None, qo=None, v=None, mode=2)),
    (-4, dict(n=2 ** 28)), (-6, dict(q=P(0x1008))), (-6, dict(cs=P(0x1004))),
    (-6, dict(ks=132)), (-6, dict(qos=516)), (-6, dict(k=P(0x1002))),
    (0, dict(n=0)), (0, dict(n=0, q=None, qo=None))])
def test_rope_status_codes(lib, want, kw):
    assert rope(lib, **kw) == want


def decode(lib, **kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, mb=4, sl=FAKE, B=2, bs=16, hq=8,
             hkv=2, d=128, fmt=0, mode=0, gs=64, sm=0.1, win=0, pre=None, cap=0.0, al=None, nb=16,
             out=FAKE, odt=0, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.fp8pa_paged_decode_attention_mod(
        a["q"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["mb"], a["sl"], a["B"], a["bs"],
        a["hq"], a["hkv"], a["d"], a["fmt"], a["mode"], a["gs"], a["sm"], a["win"], a["pre"],
        a["cap"], a["al"], a["nb"], a["out"], a["odt"], a["ws"], a["wsb"], None)


def prefill(lib, **kw):
    a = dict(q=FAKE, qo=FAKE, tq=9, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, mb=4, sl=FAKE,
             B=2, bs=16, hq=8, hkv=2, d=128, fmt=0, mode=0, gs=64, sm=0.1, win=0, pre=None,
             cap=0.0, al=None, nb=16, out=FAKE, odt=0, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.fp8pa_paged_prefill_attention(
        a["q"], a["qo"], a["tq"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["mb"], a["sl"],
        a["B"], a["bs"], a["hq"], a["hkv"], a["d"], a["fmt"], a["mode"], a["gs"], a["sm"],
        a["win"], a["pre"], a["cap"], a["al"], a["nb"], a["out"], a["odt"], a["ws"], a["wsb"],
        None)


COMMON = [
    (-1, dict(q=None)), (-1, dict(kc=None)), (-1, dict(vc=None)), (-1, dict(ks=None)),
    (-1, dict(vs=None)), (-1, dict(bt=None)), (-1, dict(sl=None)), (-1, dict(out=None)),
    (-1, dict(ws=None)), (-2, dict(fmt=3)), (-2, dict(mode=5)), (-2, dict(odt=2)),
    (-3, dict(hq=7)), (-3, dict(hkv=0)), (-3, dict(B=-1)), (-3, dict(win=-1)), (-3, dict(mb=0)),
    (-3, dict(nb=0)), (-4, dict(d=96)), (-4, dict(d=576, hkv=1, hq=64)), (-4, dict(bs=8)),
    (-4, dict(mode=2)), (-4, dict(fmt=2, mode=3, gs=32)), (-4, dict(mode=3, gs=64)),
    (-4, dict(cap=-1.0)), (-4, dict(cap=float("inf"))), (-4, dict(cap=float("nan"))),
    (-4, dict(nb=2 ** 27)), (-6, dict(q=P(0x1008))), (-6, dict(out=P(0x1004))),
    (-6, dict(ws=P(0x1001))), (0, dict(B=0))]


@pytest.mark.parametrize("want,kw", COMMON + [(-4, dict(hq=32, hkv=2))])
def test_decode_mod_status_codes(lib, want, kw):
    assert decode(lib, **kw) == want


@pytest.mark.parametrize("want,kw", COMMON + [
    (-1, dict(qo=None)), (-3, dict(tq=-1)), (-4, dict(tq=2 ** 29)), (0, dict(tq=0))])
def test_prefill_status_codes(lib, want, kw):
    assert prefill(lib, **kw) == want


def test_prefill_workspace_of_refused_sizes_is_zero(lib):
    for args in ((-1, 1, 8, 2, 128, 16, 4), (5, -1, 8, 2, 128, 16, 4), (5, 1, 7, 2, 128, 16, 4),
                 (5, 1, 8, 0, 128, 16, 4), (5, 1, 8, 2, 96, 16, 4), (2 ** 29, 1, 8, 2, 128, 16, 4),
                 (5, 1, 8, 2, 128, 0, 4), (5, 1, 8, 2, 128, 16, 0), (5, 1, 8, 2, 128, 64, 2 ** 25)):
        assert lib.fp8pa_prefill_workspace_bytes(*args) == 0


def test_wrappers_refuse_tensors_that_are_not_theirs(lib):
    """Types are looked at first, so CPU tensors show it; nothing is launched."""
    import fp8_quantised_paged_gb300 as F
    q = torch.zeros(3, 4, 64)
    i = torch.zeros(3, dtype=torch.int32)
    c = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
    s = torch.zeros(2, 2, 16, 1)
    with pytest.raises(TypeError):
        F.kv_append_rope(q, q, q, i, s, i, c, c, s, s)
    with pytest.raises(ValueError):
        F.kv_append_rope(None, q.bfloat16(), None, i, s, i, c, None, s, None)
    with pytest.raises(TypeError):
        F.paged_decode_attention_mod(q, c, c, s, s, i, i, 2, 1.0)
    with pytest.raises(ValueError):
        F.paged_decode_attention_mod(q.bfloat16(), c, c, s, s, i, i, 2, 1.0)
    with pytest.raises(TypeError):
        F.paged_prefill_attention(q, i, c, c, s, s, i, i, 2, 1.0)
    with pytest.raises(ValueError):
        F.paged_prefill_attention(q.bfloat16(), i, c, c, s, s, i, i, 2, 1.0)


@pytest.mark.gpu
def test_wrappers_refuse_shapes_that_do_not_fit(lib):
    import fp8_quantised_paged_gb300 as F
    dev = "cuda:0"
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.uint8, device=dev)
    ks = torch.zeros(2, 2, 16, 1, device=dev)
    cs = torch.zeros(10, 64, device=dev)
    ok = dict(q=bf(3, 4, 64), k=bf(3, 2, 64), v=bf(3, 2, 64), positions=i32(3), cos_sin=cs,
              slot_mapping=i32(3), k_cache=kc, v_cache=kc, k_scale=ks, v_scale=ks)
    for bad in (dict(q=bf(2, 4, 64)), dict(v=bf(3, 1, 64)), dict(positions=i32(4)),
                dict(slot_mapping=i32(2)), dict(cos_sin=cs[0]), dict(k_scale=ks[:1]),
                dict(v_cache=kc[:1]), dict(v_cache=None), dict(k=bf(3, 2, 32)),
                dict(q=bf(3, 64, 4).transpose(1, 2)), dict(q_out=bf(3, 4, 32)),
                dict(q=None, q_out=bf(3, 4, 64))):
        with pytest.raises(ValueError):
            F.kv_append_rope(**{**ok, **bad})
    ok = dict(q=bf(3, 4, 64), k_cache=kc, v_cache=kc, k_scale=ks, v_scale=ks,
              block_tables=i32(3, 2), seq_lens=i32(3), n_kv_heads=2, sm_scale=1.0)
    shared = (dict(k_cache=kc[..., :32].contiguous()), dict(v_cache=kc[:1]), dict(v_scale=None),
              dict(k_scale=ks[:1]), dict(n_kv_heads=1), dict(prefix_lens=i32(2)),
              dict(alibi_slopes=torch.zeros(3, device=dev)), dict(out=bf(3, 4, 32)),
              dict(block_tables=i32(2, 2)), dict(seq_lens=i32(4)))
    for bad in shared:
        with pytest.raises(ValueError):
            F.paged_decode_attention_mod(**{**ok, **bad})
        with pytest.raises(ValueError):
            F.paged_prefill_attention(**{**ok, "q_offsets": i32(4), **bad})
    with pytest.raises(ValueError):
        F.paged_prefill_attention(**ok, q_offsets=i32(3))
    small = torch.empty(16, dtype=torch.uint8, device=dev)
    for call, kw in ((F.paged_decode_attention_mod, {}),
                     (F.paged_prefill_attention, {"q_offsets": i32(4)})):
        with pytest.raises(F.Fp8paError):
            call(**ok, **kw, workspace=small)
