"""GPU tests of what the attention's binding refuses."""
import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
from test_tree_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [3, 20])
def test_a_mask_without_words_is_no_chain(n):
    """It would hide every drafted token; taken for no mask, it showed them."""
    c = Case([40], [n], 4, 2, 64)
    wide = c.mask.cuda()
    for mask in (wide[:, :0], torch.empty(n, 0, dtype=torch.int32, device="cuda")):
        c.mask = mask
        with pytest.raises(ValueError, match="word"):
            c.run()
    out = rarn.tree_attention(c.q[:0].cuda(), c.cache, c.table.cuda(),
                              torch.tensor(c.ctx, dtype=torch.int32, device="cuda"),
                              torch.zeros(2, dtype=torch.int32, device="cuda"), mask=wide[:0])
    assert out.shape[0] == 0
