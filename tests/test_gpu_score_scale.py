"""A score scale that is not a number makes every row NaN, with and without score modifiers."""
import pytest
import torch

from serving_ref import E4M3, INT8, MX, STATIC, TOKEN_HEAD
from test_gpu_tree import CTX, NODES, Case, F  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,mode", [(E4M3, TOKEN_HEAD), (INT8, TOKEN_HEAD), (E4M3, STATIC),
                                      (E4M3, MX)])
@pytest.mark.parametrize("mods", [{}, dict(window=40), dict(alibi=True), dict(cap=30.0)])
def test_nan(F, fmt, mode, mods):  # noqa: F811
    for d in (64, 128):
        c = Case(41, CTX, NODES, 8, 2, d, 16, fmt, mode, sm=float("nan"), **mods)
        a, kw = c.args()
        assert torch.isnan(c.run(F)).all()
        assert torch.isnan(F.paged_prefill_attention(a[0], a[1], *a[3:], **kw)).all()
        assert torch.isnan(F.paged_decode_attention_mod(a[0][:len(CTX)].contiguous(), *a[3:],
                                                        **kw))[:-1].all()
        assert F.get_device_error() == 0
