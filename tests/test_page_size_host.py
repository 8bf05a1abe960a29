"""The page size of a KVPages: checked before it is cut to 32 bits.  CPU only."""
import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn


@pytest.mark.parametrize("page_size", [0, -16, (1 << 20) + 1, (1 << 32) + 16, 1 - (1 << 32)])
def test_page_sizes_outside(page_size):
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        rarn.KVPages(i.view(1, 4), i[:1], i, i[:1], page_size)
