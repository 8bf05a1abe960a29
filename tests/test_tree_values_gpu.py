"""GPU tests of what single values and scales of the cache may do to the rows
of the attention that see them, and to those that do not."""
import pytest
import torch

import kv_ref as R
import residual_add_rmsnorm_gb300 as rarn
from test_tree_gpu import Case
from test_tree_scores_gpu import set_scores

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


def clean_rows(c):
    """Sequence 0's result without what a test plants, and its bound."""
    L = c.ctx[0] + c.new[0]
    return R.attention(c.q, *(c.values(t, s, 0, L) for t, s in ((c.cache.k, c.cache.k_scale),
                                                                (c.cache.v, c.cache.v_scale))),
                       c.visible(0), c.D ** -0.5)


# rows of 8 and of 16 to a block, 128 and 256 to a tile
SIZES = [(1, 2, 64, "e4m3"), (5, 4, 128, "e5m2"), (20, 2, 128, "e4m3"), (20, 4, 64, "e5m2"),
         (80, 2, 128, "e5m2"), (80, 2, 64, "e4m3"), (6, 2, 256, "e5m2")]


@pytest.mark.parametrize("n,G,D,fmt", SIZES)
@pytest.mark.parametrize("back", [1, 100, 249])
def test_context_values_that_are_not_finite(n, G, D, fmt, back):
    """A NaN or infinite element of a context token's value reaches every row,
    also in the tile in which the context ends."""
    c = Case([250], [n], 2 * G, 2, D, fmt=fmt, seed=30)
    want, tol = clean_rows(c)
    slots = c.slots(0, 250 + n)
    at = slots[250 - back].item()
    c.cache.v[at // 16, 0, at % 16, 3] = 0x7f if fmt == "e4m3" else 0x7e
    if fmt == "e5m2":
        c.cache.v[at // 16, 1, at % 16, 9] = 0x7c
    got = c.run().cpu()
    assert rarn.watchdog() == 0
    assert torch.isnan(got[:, :G, 3]).all()
    got[:, :G, 3] = 0
    want[:, :G, 3] = 0
    if fmt == "e5m2":      # +inf, or NaN where the weight is 0
        x = got[:, G:, 9]
        assert not torch.isfinite(x).any() and not (x < 0).any()
        got[:, G:, 9] = 0
        want[:, G:, 9] = 0
    R.check_attention(got, want, tol)


@pytest.mark.parametrize("n,G,D,fmt", SIZES)
def test_a_nan_of_no_weight(n, G, D, fmt):
    """A NaN value in keys whose weights are zero in binary32 beside later
    ones' makes its rows NaN all the same."""
    c = Case([700], [n], 2 * G, 2, D, fmt=fmt, seed=32)
    targets = torch.zeros(700 + n)
    targets[300:] = 400.0                    # log2 units
    set_scores(c, 0, targets)
    at = c.slots(0, 700)[5].item()
    c.cache.v[at // 16, 0, at % 16, 3] = 0x7f if fmt == "e4m3" else 0x7e
    got = c.run().cpu()
    assert torch.isnan(got[:, :G, 3]).all()
    got[:, :G, 3] = 0
    assert torch.isfinite(got).all()


# blocks of 8 and of 16 rows; tiles of 128 and 256 rows
ROWS = [(3, 2, 64, "e4m3"), (4, 2, 128, "e5m2"), (6, 2, 128, "e4m3"), (6, 2, 96, "e4m3"),
        (12, 3, 192, "e4m3"), (6, 2, 256, "e5m2"), (20, 2, 128, "e4m3"), (40, 2, 64, "e5m2"),
        (80, 2, 128, "e4m3"), (90, 2, 64, "e4m3")]


@pytest.mark.parametrize("n,G,D,fmt", ROWS)
@pytest.mark.parametrize("ctx", [0, 5, 200])
@pytest.mark.parametrize("power", [40, 90])
def test_a_hidden_value_scale(n, G, D, fmt, ctx, power):
    """A drafted token with a finite value scale far over all others' (what a
    slot that was left out still holds): the rows that do not see it are as if
    it were not there, those that see it are right too."""
    c = Case([ctx], [n], 2 * G, 2, D, fmt=fmt, seed=50)
    want, tol = clean_rows(c)
    at = c.slots(0, ctx + n)[ctx + n // 2].item()
    c.cache.v_scale[at // 16, :, at % 16] = 2.0 ** power
    got, vis = c.run().cpu(), c.visible(0)
    assert rarn.watchdog() == 0
    sees = vis[:, ctx + n // 2]
    assert sees.any() and not sees.all()
    R.check_attention(got[~sees], want[~sees], tol[~sees])
    c.check(got)
