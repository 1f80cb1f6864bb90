"""Prefills as a server issues them: one long chunk among single tokens, and block
tables far wider than the requests, up to where tiles are no longer converted once."""
import pytest
import torch

import serving_ref as R
from test_gpu_prefill import DEV, F, LONG, Batch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("singles", [3, 40])
@pytest.mark.parametrize("reach", [0, 4096])
@pytest.mark.parametrize("mods", [{}, {"window": 50, "cap": 20.0}])
def test_a_long_chunk_among_single_tokens(F, singles, reach, mods):  # noqa: F811
    """4000 rows and `singles` times 8: a mean above and below 768 rows a request."""
    lens = [700] + [37 + 13 * i % 400 for i in range(singles)]
    b = Batch(lens, [500] + [1] * singles, 8, 1, 128, 16, R.E4M3, R.TOKEN_HEAD, seed=43,
              reach=reach)
    ref = b.ref(device=DEV, **mods)
    got = b.run(F, **mods)
    R.check(got, ref, 128, half=R.TOKEN_HEAD, cap=mods.get("cap", 0.0))
    assert F.get_device_error() == 0


@pytest.mark.parametrize("over", [False, True])
def test_tables_that_reach_past_what_is_converted_once(F, over):  # noqa: F811
    """Long chunks whose tables reach 262144 tokens in all (1 GiB of tiles at 8 KV
    heads of 128 dims), and one page more."""
    batch, bs, d, hkv = 2, 64, 128, 8
    reach = 131072 + (bs if over else 0)
    b = Batch([300, 130], [100, 130], LONG // 8 * hkv, hkv, d, bs, R.E4M3, R.TOKEN_HEAD, seed=44,
              reach=reach)
    need = F.prefill_workspace_bytes(230, batch, b.hq, hkv, d, bs, b.bt.shape[1])
    assert (need < 1 << 30) == over
    ref = b.ref(device=DEV)
    R.check(b.run(F), ref, d, half=R.TOKEN_HEAD)
    assert F.get_device_error() == 0
