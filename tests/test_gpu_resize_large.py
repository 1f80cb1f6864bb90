"""A resize that asks for more pages than 32 bits count."""
import pytest
import torch

from pages_ref import NO_BLOCK
from test_pages_refusals import call, lib  # noqa: F401

DEV = "cuda:0"


def test_pools_whose_size_plus_one_passes_32_bits_are_refused(lib):  # noqa: F811
    for which in ("fork", "resize", "compact", "keep"):
        # (sizes are looked at before pointers: without tables nothing is launched either way)
        assert call(lib, which, nb=2 ** 31 - 1, bs=1, bt=None) == -4


@pytest.mark.gpu
def test_growth_past_32_bits_finds_no_page():
    """2053 rows of 2^20 pages each, of a pool of 2^30 pages of one token with 10 free ones (17
    GB of tables, counts and workspace)."""
    import fp8_quantised_paged_gb300 as F
    F.get_device_error()
    rows, cols, nb = 2053, 2 ** 20, 2 ** 30
    t = torch.empty(rows, cols, dtype=torch.int32, device=DEV)
    t[-1, :10] = -1
    n = torch.zeros(rows, dtype=torch.int32, device=DEV)
    r = torch.ones(nb, dtype=torch.int32, device=DEV)
    free = torch.tensor([3, 5, 1000, 10 ** 6, 10 ** 6 + 1, 10 ** 7, 2 ** 29, 2 ** 29 + 7, 2 ** 30 - 2,
                         2 ** 30 - 1], device=DEV)
    r[free] = 0
    then = torch.full_like(n, cols)
    F.kv_resize(then, t, n, r, 1)
    assert F.get_device_error() == NO_BLOCK
    assert not n.any()
    assert int((r == 0).sum()) == 10 and not r[free].any()
    # one row that fits, ahead of them
    then[0] = 10
    F.kv_resize(then, t, n, r, 1)
    assert F.get_device_error() == NO_BLOCK
    assert int(n[0]) == 10 and not n[1:].any()
    assert t[0, :10].tolist() == free.tolist()
    assert bool((r == 1).all())
