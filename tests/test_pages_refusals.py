"""Refused arguments of the page operators: status codes and exceptions, none of which
touches a device."""
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


def arrays(ptrs, each):
    n = len(ptrs)
    a = (P * n)(*ptrs)
    b = (ctypes.c_longlong * n)(*each)
    return ctypes.cast(a, P), ctypes.cast(b, P), n, (a, b)


def call(lib, which, **kw):
    pages, sizes, n, keep = arrays(kw.pop("ptrs", (0x1000, 0x2000)), kw.pop("each", (2048, 128)))
    a = dict(acc=FAKE, ma=4, off=FAKE, bt=FAKE, mb=4, sl=P(0x4000), B=3, pages=pages, sizes=sizes,
             n=n, hkv=2, nb=8, bs=16, nl=P(0x8000), src=FAKE, dst=FAKE, f=2, ref=FAKE, map=FAKE,
             ws=FAKE, wsb=1 << 20)
    a.update(kw)
    g = lambda *k: [a[x] for x in k]  # noqa: E731
    if which == "keep":
        return lib.fp8pa_kv_keep_accepted(*g("acc", "ma", "off", "bt", "mb", "sl", "B", "pages",
                                             "sizes", "n", "hkv", "nb", "bs", "nl"), None)
    if which == "fork":
        return lib.fp8pa_kv_fork(*g("src", "dst", "f", "bt", "mb", "sl", "B", "ref", "pages",
                                    "sizes", "n", "nb", "bs", "ws", "wsb"), None)
    if which == "resize":
        return lib.fp8pa_kv_resize(*g("nl", "bt", "mb", "sl", "B", "ref", "nb", "bs", "ws", "wsb"),
                                   None)
    return lib.fp8pa_kv_compact(*g("bt", "mb", "sl", "B", "ref", "pages", "sizes", "n", "nb", "bs",
                                   "map", "ws", "wsb"), None)


ROWS = [(-1, dict(bt=None)), (-1, dict(sl=None)), (-3, dict(B=-1)), (-3, dict(mb=0)),
        (-3, dict(nb=0)), (-3, dict(bs=0)), (-4, dict(nb=2 ** 27)), (-4, dict(mb=2 ** 21))]
ARRAYS = [(-1, dict(pages=None)), (-1, dict(sizes=None)), (-1, dict(ptrs=(0x1000, None))),
          (-3, dict(n=-1)), (-3, dict(each=(2048, 0))), (-4, dict(each=(2 ** 31, 128))),
          (-6, dict(ptrs=(0x1008, 0x2000))), (-6, dict(each=(2048, 72)))]
SCRATCH = [(-1, dict(ws=None)), (-5, dict(wsb=40)), (-6, dict(ws=P(0x1002))), (-1, dict(ref=None))]


@pytest.mark.parametrize("want,kw", ROWS + ARRAYS + [
    (-1, dict(acc=None)), (-1, dict(off=None)), (-1, dict(nl=None)), (-3, dict(ma=0)),
    (-3, dict(hkv=0)), (-3, dict(each=(2048, 16 * 9))), (-4, dict(nl=P(0x4000))),
    (-4, dict(nl=P(0x4008))), (-4, dict(ma=2 ** 26)), (0, dict(B=0))])
def test_keep_status_codes(lib, want, kw):
    assert call(lib, "keep", **kw) == want


@pytest.mark.parametrize("want,kw", ROWS + ARRAYS + SCRATCH + [
    (-1, dict(src=None)), (-1, dict(dst=None)), (-3, dict(f=-1)), (-3, dict(f=4)),
    (0, dict(f=0))])
def test_fork_status_codes(lib, want, kw):
    assert call(lib, "fork", **kw) == want


@pytest.mark.parametrize("want,kw", ROWS + SCRATCH + [
    (-1, dict(nl=None)), (-4, dict(nl=P(0x4004))), (0, dict(B=0))])
def test_resize_status_codes(lib, want, kw):
    assert call(lib, "resize", **kw) == want


@pytest.mark.parametrize("want,kw", ROWS + ARRAYS + SCRATCH + [(-1, dict(map=None))])
def test_compact_status_codes(lib, want, kw):
    assert call(lib, "compact", **kw) == want


def test_workspace_size(lib):
    assert lib.fp8pa_pages_workspace_bytes(10, 100) >= 4 * 100
    assert lib.fp8pa_pages_workspace_bytes(-1, 100) == 0
    assert lib.fp8pa_pages_workspace_bytes(10, 0) == 0


def test_wrappers_refuse_tensors_that_are_not_theirs(lib):
    import fp8_quantised_paged_gb300 as F
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        F.KvPages([])
    with pytest.raises(ValueError):
        F.KvPages([torch.zeros(4, 2, 16, 64)])  # not on a CUDA device
    with pytest.raises(ValueError):
        F.kv_resize(i, i, i, i, 16)
    with pytest.raises(F.Fp8paError):
        F.pages_workspace_bytes(-1, 4)


@pytest.mark.gpu
def test_wrappers_refuse_shapes_that_do_not_fit(lib):
    import fp8_quantised_paged_gb300 as F
    dev = "cuda:0"
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=dev)  # noqa: E731
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device=dev)  # noqa: E731
    c = u8(4, 2, 16, 64)
    for bad in ([c, u8(5, 2, 16, 64)], [c, u8(4, 2, 32, 64)], [c, u8(4, 64).t()], [u8(4)]):
        with pytest.raises(ValueError):
            F.KvPages(bad)
    per_page = F.KvPages([c, torch.zeros(4, 4, device=dev)])
    pages = F.KvPages([c])
    t, n, r = i32(3, 2), i32(3), i32(4)
    keep = dict(accepted=i32(3, 2), q_offsets=i32(4), block_tables=t, seq_lens=n, pages=pages)
    for bad in (dict(accepted=i32(2, 2)), dict(accepted=i32(3)), dict(q_offsets=i32(3)),
                dict(seq_lens=i32(2)), dict(pages=per_page), dict(new_lens=i32(2)),
                dict(pages=F.KvPages([u8(4, 64)]))):
        with pytest.raises(ValueError):
            F.kv_keep_accepted(**{**keep, **bad})
    with pytest.raises(TypeError):
        F.kv_keep_accepted(**{**keep, "accepted": i32(3, 2).long()})
    fork = dict(src_rows=i32(1), dst_rows=i32(1), block_tables=t, seq_lens=n, ref_counts=r,
                pages=per_page)
    for bad in (dict(dst_rows=i32(2)), dict(ref_counts=i32(5)), dict(block_tables=i32(2, 2))):
        with pytest.raises(ValueError):
            F.kv_fork(**{**fork, **bad})
    with pytest.raises(F.Fp8paError):
        F.kv_fork(**{**fork, "workspace": u8(4)})
    with pytest.raises(ValueError):
        F.kv_resize(i32(2), t, n, r, 16)
    with pytest.raises(ValueError):
        F.kv_compact(t, n, i32(3), pages)
    with pytest.raises(ValueError):
        F.kv_compact(t, n, r, pages, page_map=i32(3))
