"""Arguments that the serving calls of the binding refuse before anything reaches the
library (CPU only)."""
import pytest
import torch

from shared_prefix_fan_gb300 import binding


@pytest.mark.parametrize("page", [1, 17])
def test_copy_pages_q4_refuses_pages_it_would_copy_in_part(page):
    """A page is copied as pairs of 72-byte rows: with an odd size its last row, or all of a
    page of one, would stay behind."""
    pool = torch.zeros((2, 1, page * 72), dtype=torch.uint8)
    with pytest.raises(ValueError, match="page_size"):
        binding.copy_pages_q4(pool, pool, torch.zeros((1, 2), dtype=torch.int32), page)
