"""Arrays of a KvPages are each given once."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_arrays_that_overlap_are_refused():
    import fp8_quantised_paged_gb300 as F
    c = torch.zeros(9, 2, 16, 64, dtype=torch.uint8, device="cuda:0")
    other = torch.zeros(8, 2, 16, 1, device="cuda:0")
    for bad in ([c, c], [c[:8], other, c[1:]], [c[1:], c[:8]], [other, other.view(8, 2, 16, 1)],
                [c[:8], c[:8].view(8, 2, 16, 8, 8)]):
        with pytest.raises(ValueError, match="overlap"):
            F.KvPages(bad)


def test_arrays_of_one_buffer_are_taken():
    """Layers that lie one behind the other in one tensor."""
    import fp8_quantised_paged_gb300 as F
    c = torch.zeros(6, 8, 2, 16, 64, dtype=torch.uint8, device="cuda:0")
    assert F.KvPages(c.unbind()).num_blocks == 8
    assert F.KvPages(list(reversed(c.unbind()))).per_token
