"""The prefill's workspace query refuses what the call refuses."""
import pytest

from test_serving_refusals import lib, prefill  # noqa: F401

pytestmark = pytest.mark.gpu  # the query asks the device


@pytest.mark.parametrize("kw", [
    {}, dict(tq=0), dict(B=0), dict(bs=32), dict(bs=64, d=64), dict(hq=600, hkv=3),
    dict(bs=8), dict(bs=1), dict(bs=48), dict(bs=128), dict(d=96), dict(hq=7), dict(mb=0),
    dict(mb=2 ** 27), dict(mb=2 ** 26), dict(mb=2 ** 26, hkv=1, hq=4),
    dict(tq=2 ** 26, mb=2 ** 20), dict(tq=2 ** 22, B=2 ** 18, mb=2 ** 16)])
def test_sizes_that_are_refused_need_no_workspace(lib, kw):  # noqa: F811
    a = dict(tq=9, B=2, hq=8, hkv=2, d=128, bs=16, mb=4)
    a.update(kw)
    need = lib.fp8pa_prefill_workspace_bytes(a["tq"], a["B"], a["hq"], a["hkv"], a["d"], a["bs"],
                                             a["mb"])
    # nothing is launched: behind the sizes, a null pointer stops the call
    got = prefill(lib, **kw, q=None)
    assert (need == 0) == (got in (-3, -4)), (need, got)
