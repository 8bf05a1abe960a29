"""GPU tests of the attention over the 8-bit cache for a prompt's chunk: some
hundreds of new tokens without a mask, in many blocks of rows and, behind the
context, whole tiles that a block does not see."""
import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
from test_tree_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctx,new,G,D,dt,page", [
    ([77], [500], 2, 128, "bf16", 16), ([0], [260], 4, 64, "f16", 64),
    ([0, 300, 5], [129, 1, 200], 2, 128, "bf16", 24), ([40], [300], 1, 192, "bf16", 16),
    ([0], [200], 2, 256, "f16", 8), ([130, 0], [90, 131], 2, 96, "bf16", 7)])
def test_a_prompts_chunk(ctx, new, G, D, dt, page):
    c = Case(ctx, new, 2 * G, 2, D, dt=dt, page=page, seed=70, mask="chain")
    out = c.run()
    assert rarn.watchdog(clear=True) == 0
    c.check(out)
    assert torch.equal(c.run(out=torch.zeros_like(out)), out)
