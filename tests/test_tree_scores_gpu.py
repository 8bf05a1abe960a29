"""GPU tests of the attention over the 8-bit cache where a row's scores rise so
steeply that what it has summed up is scaled down, against binary64."""
import math

import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
from test_tree_gpu import Case

pytestmark = pytest.mark.gpu

ONE = {"e4m3": 0x38, "e5m2": 0x3c}


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


def set_scores(c, b, targets):
    """Key j of sequence b scores about targets[j] (in log2 units) against
    every row: keys of ones, their scales the rest, queries near one."""
    g = torch.Generator().manual_seed(5)
    c.q = (1 + 0.02 * torch.randn(c.q.shape, generator=g)).to(c.dt)
    at = c.slots(b, len(targets)).cuda()
    page, slot = at // c.page, at % c.page
    c.cache.k[page, :, slot] = ONE[c.fmt]
    c.cache.k_scale[page, :, slot] = (targets.float() * math.log(2) / c.D ** 0.5).cuda()[:, None]


MANY = [(20, 2, 128, "bf16", "e4m3"), (40, 1, 64, "f16", "e5m2"), (80, 2, 128, "bf16", "e4m3"),
        (80, 2, 64, "f16", "e4m3"), (80, 2, 128, "f16", "e5m2"), (3, 2, 128, "bf16", "e4m3")]


@pytest.mark.parametrize("n,G,D,dt,fmt", MANY)
def test_the_second_half_of_a_pass_has_the_largest_score(n, G, D, dt, fmt):
    """In every 64 keys one of the last 32 scores 2^13 above all before it, and
    its value is zero, so that the result is what the others' weights come to
    after they are scaled down: a bound relative to their sum."""
    L = 640 + n
    c = Case([640], [n], 2 * G, 2, D, dt=dt, fmt=fmt, seed=12)
    j = torch.arange(L)
    g = torch.Generator().manual_seed(1)
    targets = 13.0 * (j // 64) - 2 * torch.rand(L, generator=g)
    high = j % 64 == 40
    targets[high] += 14
    set_scores(c, 0, targets)
    at = c.slots(0, L)[high].cuda()
    c.cache.v[at // c.page, :, at % c.page] = 0
    out = c.run()
    assert rarn.watchdog() == 0
    c.check(out)
    assert torch.equal(c.run(out=torch.zeros_like(out)), out)
