"""The prefill's softmax sums where V is zero or its scales are extreme."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_gpu_prefill import DEV, F, Batch  # noqa: F401

pytestmark = pytest.mark.gpu

KINDS = [(R.E4M3, R.MX, 32), (R.E5M2, R.MX, 16), (R.E4M3, R.TOKEN_HEAD, 32),
         (R.INT8, R.TOKEN_HEAD, 32), (R.E5M2, R.TOKEN_HEAD, 32), (R.E4M3, R.SEGMENT, 32)]


def check(b, F, mode, extra=0.0, **mods):  # noqa: F811
    """Against the reference.  A token's exponent in P is z - reference + e, e its V
    group's exponent; |e| <= 128 rounds to 2^-18 there, twice in the quotient of P and
    sum: 2^-17 of A more, and 2^-17 more for the hardware exponential's own error at
    such arguments."""
    out, A, Z, B, W, Fl = b.ref(device=DEV, **mods)
    R.check(b.run(F, **mods), (out, A, Z, B, W + 2.0 ** -16 * A + extra, Fl), b.d, half=mode)
    assert F.get_device_error() == 0


@pytest.mark.parametrize("fmt,mode,gs", KINDS)
@pytest.mark.parametrize("chunk", [80, 96])  # 640 and 768 rows: converted by each block, and once
@pytest.mark.parametrize("d", [64, 128])
def test_a_long_span_of_zero_values_ahead_of_others(F, fmt, mode, gs, chunk, d):  # noqa: F811
    """Tokens whose V is zero and whose scale is the smallest that the mode holds take
    part in the sums of every row: 3500 of 4000 tokens, about 20 tiles to a range, and
    near-equal scores, so that their weights add up."""
    zero, n = 3500 // 64 * 64, 4000
    b = Batch([n] * 4, [chunk] * 4, 64, 8, d, 64, fmt, mode, gs, seed=30, qgain=0.01)
    _, vc, _, vs = b.cache
    first = b.bt[:, :zero // 64].flatten().long()  # whole blocks
    vc[first] = 128 if fmt == R.INT8 else 0
    vs[first] = 0
    check(b, F, mode)


@pytest.mark.parametrize("fmt,mode,gs", KINDS)
@pytest.mark.parametrize("chunk", [80, 96])
@pytest.mark.parametrize("up", [-60, 60, 100])
def test_values_of_every_magnitude(F, fmt, mode, gs, chunk, up):  # noqa: F811
    """All of V times 2^up."""
    b = Batch([700, 300], [chunk, chunk], 8, 1, 128, 16, fmt, mode, gs, seed=31)
    vs = b.cache[3]
    if mode == R.MX:
        vs += up
    else:
        vs *= 2.0 ** up
    check(b, F, mode)


@pytest.mark.parametrize("chunk", [80, 96])
@pytest.mark.parametrize("up", [-90, -110])
def test_the_smallest_values(F, chunk, up):  # noqa: F811
    """Below 2^-94 a value is off by up to half of 2^-104, V^'s smallest step."""
    b = Batch([700, 300], [chunk, chunk], 8, 1, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=32)
    b.cache[3] *= 2.0 ** up
    check(b, F, R.TOKEN_HEAD, extra=2.0 ** -105)
