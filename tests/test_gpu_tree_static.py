"""Tree attention with static channel scales: how well q times the scales is kept.

Tolerance (stated before any run).  q c, with c the channel's scale, is one fp32 product
(2^-24).  FP8 codes meet it as three E4M3 terms.  Of an element of exponent e the first is off
by at most half a step, 2^(e - 4); what it leaves is 2^(e - 4) itself, which is exact, or has
an exponent of at most e - 5, so the second leaves at most 2^(e - 9), and the third 2^(e - 14).
All stop at half of E4M3's smallest step: 2^-17 of the row's largest element, as for other
scales.  So an element is off by 2^-14 of itself and that, where tree_ref.py allows 2^-9.
INT8 codes meet it as f16, 2^-11.  The rest is tree_ref.py's bound.
"""
import pytest
import torch

from serving_ref import E4M3, E5M2, INT8, STATIC
from test_gpu_tree import CTX, DEV, NODES, Case, F  # noqa: F401
from tree_ref import check_tree

pytestmark = pytest.mark.gpu


def tight(ref, fmt):
    out, A, Z, B, W, Fl = ref
    own = 2.0 ** -11 if fmt == INT8 else 2.0 ** -14 + 2.0 ** -24
    return out, A, Z, B, W, Fl - (2.0 ** -9 - own) * Z


def check(F, c, what=""):  # noqa: F811
    ref = tight(c.ref(), c.fmt)
    for dt in (torch.float32, torch.bfloat16):
        out = c.run(F, out_dtype=dt)
        assert F.get_device_error() == 0
        check_tree(out, ref, c.d, dt == torch.bfloat16, c.cap, what)


@pytest.mark.parametrize("fmt", [E4M3, E5M2, INT8])
@pytest.mark.parametrize("d,bs,hq,hkv", [(128, 16, 16, 2), (64, 32, 12, 4), (128, 64, 3, 1)])
@pytest.mark.parametrize("mods", [{}, dict(alibi=True), dict(cap=30.0, window=40)])
def test_random_scales(F, fmt, d, bs, hq, hkv, mods):  # noqa: F811
    c = Case(31, CTX, NODES, hq, hkv, d, bs, fmt, STATIC, **mods)
    check(F, c)
    c.sm *= 4  # sharper weights
    check(F, c)


@pytest.mark.parametrize("fmt,code", [(E4M3, 0x38), (E5M2, 0x3C)])  # the code of 1.0
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scales_that_two_terms_round_alike(F, fmt, code, d, sign):  # noqa: F811
    """Even tokens have codes in the first half of the dims only, odd ones in the second; the
    scales of a half are all rounded the same way where two terms hold them, those of the other
    half the other way, so that the two kinds' scores part."""
    c = Case(32, [500, 90], [9, 30], 8, 2, d, 16, fmt, STATIC, sm=40.0 / d)
    kc, vc, ks, vs = c.cache
    # 1 + 2^-4 - 2^-8 -+ 2^-9: of 2^-4 - 2^-8 -+ 2^-9 the nearest E4M3 (steps of 2^-8) is as
    # far as it can be
    near = 2.0 ** -9 * (1 - 2.0 ** -6)
    up, down = 1 + 2.0 ** -4 - 2.0 ** -8 - near, 1 + 2.0 ** -4 - 3 * 2.0 ** -8 + near
    ks.copy_(torch.where(torch.arange(d, device=DEV) < d // 2, up, down).expand_as(ks))
    kc.zero_()
    kc[:, :, 0::2, :d // 2] = code
    kc[:, :, 1::2, d // 2:] = code
    vc[:, :, 0::2], vc[:, :, 1::2] = code, code | 0x80
    vs.fill_(1.0)
    c.q.fill_(sign)
    check(F, c, "alike")


def test_scales_far_apart(F):  # noqa: F811
    """Channels of scales 2^-30 to 2^30 of one another, with codes that undo them."""
    for fmt in (E4M3, E5M2):
        c = Case(33, [300], [20], 8, 2, 128, 16, fmt, STATIC)
        ks = c.cache[2]
        f = torch.exp2(torch.arange(128, device=DEV) % 61 - 30.0)
        ks.mul_(f)
        c.q.copy_((c.q.float() / f).bfloat16())
        check(F, c)
