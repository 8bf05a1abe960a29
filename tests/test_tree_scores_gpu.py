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


def set_exact_scores(c, b, targets, scale, sign=1):
    """Key j of sequence b scores targets[j] / log2(e) / D ** 0.5 exactly
    (products of powers of two; targets in binary32) against every row."""
    c.q = torch.full(c.q.shape, float(scale)).to(c.dt)
    at = c.slots(b, len(targets)).cuda()
    page, slot = at // c.page, at % c.page
    c.cache.k[page, :, slot] = ONE[c.fmt] | (0 if sign > 0 else 0x80)
    c.cache.k_scale[page, :, slot] = targets.float().cuda()[:, None]


@pytest.mark.parametrize("n,G,D,dt,fmt", [(3, 2, 64, "bf16", "e4m3"), (20, 2, 128, "bf16", "e5m2"),
                                          (80, 2, 64, "bf16", "e4m3")])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_magnitude(n, G, D, dt, fmt, sign):
    """Scores so large that every weight but the largest's is zero: the result
    is the mean of the values that tie for it.  Over magnitudes of scores and
    of value scales, with the largest among the first keys, rising from key to
    key, or the same for all."""
    L = 300 + n
    c = Case([300], [n], 2 * G, 2, D, dt=dt, fmt=fmt, seed=20)
    at = c.slots(0, L).cuda()
    vis = c.visible(0)
    j = torch.arange(L, dtype=torch.float64)
    shapes = {"first": torch.where(j % 29 == 3, 1.0, 0.5 + (j % 7) / 32),
              "rising": (j + 200) / 512, "same": torch.ones(L, dtype=torch.float64)}
    x = c.values(c.cache.v, torch.ones_like(c.cache.v_scale), 0, L)
    for e in (24, 28, 29, 34, 60):
        for vs in (-16, -14, -13, 0, 10, 16, 20, 60):
            for name, shape in shapes.items():
                if sign < 0:
                    shape = 1.25 - shape      # the order of -shape, positive scales
                set_exact_scores(c, 0, shape * 2.0 ** (e // 2), 2.0 ** (e - e // 2), sign)
                c.cache.v_scale[at // c.page, :, at % c.page] = 2.0 ** vs
                out = c.run().cpu().double()
                t = (sign * shape).float()[None].expand(n, L).masked_fill(~vis, -math.inf)
                w = (t == t.amax(-1, keepdim=True)).double()
                w /= w.sum(-1, keepdim=True)
                v = x * 2.0 ** vs
                v = v.repeat_interleave(G, 1)
                want, mag = (torch.einsum("ij,jhd->ihd", w, y) for y in (v, v.abs()))
                # weights in binary16, of value scales down to 2^-10 of its units
                # normal, or subnormal with 8 bits; sums in binary32; one rounding
                tol = 2.0 ** -8 * mag + 2.0 ** -8 * want.abs() + 1e-30
                bad = ~((out - want).abs() <= tol)
                assert not bad.any(), (name, e, vs, int(bad.sum()))
    assert rarn.watchdog() == 0
