"""Refused arguments of the tree attention: status codes and exceptions, none of which
touches a device; and the wrapper of kv_resize, whose device is its counts'."""
import pytest
import torch

from test_serving_refusals import COMMON, FAKE, P, lib  # noqa: F401


def tree(lib, **kw):  # noqa: F811
    a = dict(q=FAKE, qo=FAKE, tq=9, pa=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, mb=4,
             sl=FAKE, B=2, bs=16, hq=8, hkv=2, d=128, fmt=0, mode=0, gs=64, sm=0.1, win=0,
             pre=None, cap=0.0, al=None, nb=16, out=FAKE, odt=0, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return lib.fp8pa_paged_tree_attention(
        a["q"], a["qo"], a["tq"], a["pa"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["mb"],
        a["sl"], a["B"], a["bs"], a["hq"], a["hkv"], a["d"], a["fmt"], a["mode"], a["gs"], a["sm"],
        a["win"], a["pre"], a["cap"], a["al"], a["nb"], a["out"], a["odt"], a["ws"], a["wsb"],
        None)


# 2^22 rows of one request are 2^15 blocks of 128: with two KV heads and 2^15 tiles (tables of
# 2^18 pages) the planner's units pass 2^31, which blocks of 256 rows would not
UNITS = dict(hq=2, hkv=2, tq=2 ** 22, B=1)


@pytest.mark.parametrize("want,kw", COMMON + [
    (-1, dict(qo=None)), (-1, dict(pa=None)), (-3, dict(tq=-1)), (-4, dict(tq=2 ** 29)),
    (-4, dict(**UNITS, mb=2 ** 18)), (-1, dict(**UNITS, mb=2 ** 17, q=None)),
    (0, dict(tq=0)), (0, dict(tq=0, pa=None)), (0, dict(B=0, pa=None))])
def test_tree_status_codes(lib, want, kw):  # noqa: F811
    assert tree(lib, **kw) == want


def test_tree_workspace_of_refused_sizes_is_zero(lib):  # noqa: F811
    for args in ((-1, 1, 8, 2, 128, 16, 4), (5, -1, 8, 2, 128, 16, 4), (5, 1, 7, 2, 128, 16, 4),
                 (5, 1, 8, 0, 128, 16, 4), (5, 1, 8, 2, 96, 16, 4), (2 ** 29, 1, 8, 2, 128, 16, 4),
                 (5, 1, 8, 2, 128, 0, 4), (5, 1, 8, 2, 128, 16, 0), (5, 1, 8, 2, 128, 64, 2 ** 25),
                 (2 ** 22, 1, 2, 2, 128, 16, 2 ** 18)):
        assert lib.fp8pa_tree_workspace_bytes(*args) == 0


@pytest.mark.gpu  # the query asks the device
@pytest.mark.parametrize("kw", [
    {}, dict(tq=0), dict(B=0), dict(bs=32), dict(bs=64, d=64), dict(hq=600, hkv=3), dict(bs=8),
    dict(bs=48), dict(d=96), dict(hq=7), dict(mb=0), dict(mb=2 ** 27),
    dict(**UNITS, mb=2 ** 17), dict(**UNITS, mb=2 ** 18)])
def test_sizes_that_are_refused_need_no_workspace(lib, kw):  # noqa: F811
    a = dict(tq=9, B=2, hq=8, hkv=2, d=128, bs=16, mb=4)
    a.update(kw)
    need = lib.fp8pa_tree_workspace_bytes(a["tq"], a["B"], a["hq"], a["hkv"], a["d"], a["bs"],
                                          a["mb"])
    assert (need == 0) == (tree(lib, **kw, q=None) in (-3, -4)), need


def test_wrappers_refuse_tensors_that_are_not_theirs(lib):  # noqa: F811
    """Types are looked at first, so CPU tensors show it; nothing is launched."""
    import fp8_quantised_paged_gb300 as F
    q = torch.zeros(3, 4, 64)
    i = torch.zeros(3, dtype=torch.int32)
    c = torch.zeros(2, 2, 16, 64, dtype=torch.uint8)
    s = torch.zeros(2, 2, 16, 1)
    with pytest.raises(TypeError):
        F.paged_tree_attention(q, i, i, c, c, s, s, i, i, 2, 1.0)
    with pytest.raises(ValueError):
        F.paged_tree_attention(q.bfloat16(), i, i, c, c, s, s, i, i, 2, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        F.kv_resize(i, i.view(3, 1), i, i, 16)


@pytest.mark.gpu
def test_wrappers_refuse_shapes_that_do_not_fit(lib):  # noqa: F811
    import fp8_quantised_paged_gb300 as F
    dev = "cuda:0"
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device=dev)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    kc = torch.zeros(2, 2, 16, 64, dtype=torch.uint8, device=dev)
    ks = torch.zeros(2, 2, 16, 1, device=dev)
    ok = dict(q=bf(3, 4, 64), q_offsets=i32(4), parents=i32(3), k_cache=kc, v_cache=kc,
              k_scale=ks, v_scale=ks, block_tables=i32(3, 2), seq_lens=i32(3), n_kv_heads=2,
              sm_scale=1.0)
    for bad in (dict(q=bf(3, 256)), dict(q=bf(4, 3, 64).transpose(0, 1)), dict(q_offsets=i32(3)),
                dict(parents=i32(2)), dict(k_cache=kc[..., :32].contiguous()),
                dict(v_cache=kc[:1]), dict(v_scale=None), dict(v_cache=None),
                dict(k_scale=ks[:1]), dict(n_kv_heads=1), dict(prefix_lens=i32(2)),
                dict(alibi_slopes=torch.zeros(3, device=dev)), dict(out=bf(3, 4, 32)),
                dict(block_tables=i32(2, 2)), dict(seq_lens=i32(4)), dict(parents=i32(3).cpu())):
        with pytest.raises(ValueError):
            F.paged_tree_attention(**{**ok, **bad})
    for bad in (dict(parents=i32(3).long()), dict(q_offsets=i32(4).float()),
                dict(out=bf(3, 4, 64).half())):
        with pytest.raises(TypeError):
            F.paged_tree_attention(**{**ok, **bad})
    for bad in (dict(workspace=torch.empty(16, dtype=torch.uint8, device=dev)), dict(window=-1),
                dict(logit_cap=-1.0), dict(fmt=7)):
        with pytest.raises(F.Fp8paError):
            F.paged_tree_attention(**{**ok, **bad})
    with pytest.raises(F.Fp8paError):
        F.tree_workspace_bytes(3, 3, 4, 2, 96, 16, 2)
