"""GPU tests of the verification at the edges of its definition: draws that end exactly on a
border, probabilities outside 0 .. 1 in the tests of drafts, drafts that are no tokens."""
import random

import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
from test_verify_gpu import run

pytestmark = pytest.mark.gpu

INDEX_BIT = 16
NAN, INF = float("nan"), float("inf")


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


def halves(units):
    """A weight of `units` 2^-46 as two binary32 numbers, both not zero."""
    low = units & (1 << 22) - 1
    return [(units - low) * 2.0 ** -46, low * 2.0 ** -46]


def borders(count, seed):
    """(u, total, the whole part of u total) whose product a binary64 multiplication that
    rounds to nearest lifts to the next whole number; in units of 2^-24 and 2^-46."""
    r, got = random.Random(seed), [(10402440, 60473987187256)]
    while len(got) < count:
        u, total = r.randrange(1 << 23, 1 << 24), r.randrange(1 << 45, 1 << 46)
        if int(u * 2.0 ** -24 * float(total)) > u * total >> 24:
            got.append((u, total))
    return [(u, t, u * t >> 24) for u, t in got]


def test_a_draw_that_ends_on_a_border():
    rows, want, numbers = [], [], []
    for u, total, whole in borders(150, 1):
        # the first two tokens' weight is just more than u total, or just not
        for first, token in ((whole + 1, 1), (whole, 2)):
            if first % (1 << 22) == 0 or (total - first) % (1 << 22) == 0:
                continue
            rows.append(halves(first) + halves(total - first))
            want.append(token)
            numbers.append(u * 2.0 ** -24)
    B = len(rows)
    got = run(torch.tensor(rows), [0] * B, list(range(B + 1)), torch.zeros(B),
              torch.tensor(numbers), 0)
    assert got[0] == [[w] for w in want]
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16])
def test_drafts_are_tested_by_values_of_0_to_1(dt):
    """u q < p with both taken as 0 .. 1 and NaN as 0."""
    cases = [(p, q, u) for p in (0.0, 0.25, 1.0, 2.0, -1.0, NAN, INF, -INF)
             for q in (0.0, 0.5, 1.0, 3.0, -0.5, NAN, INF, -INF) for u in (0.0, 0.25, 0.75)]

    def unit(x):
        return min(max(x, 0.0), 1.0) if x == x else 0.0

    # token 1 is drafted; token 0 can always be drawn
    probs = torch.tensor([[0.5, p] if row == 0 else [0.5, 0.25]
                          for p, q, u in cases for row in (0, 1)], dtype=dt)
    drafts = torch.tensor([[0.0, q] for p, q, u in cases for row in (0, 1)], dtype=dt)
    B = len(cases)
    got = run(probs, [0, 1] * B, list(range(0, 2 * B + 1, 2)),
              torch.tensor([u for p, q, u in cases for row in (0, 1)]), torch.zeros(B), 1, drafts)
    for (p, q, u), n in zip(cases, got[2]):
        assert n == (2 if u * unit(q) < unit(p) else 1), (p, q, u)


@pytest.mark.parametrize("token", [-1, 3, 2 ** 40])
def test_a_draft_that_is_no_token_takes_nothing(token):
    """Behind it the target's own row is drawn from, whatever the drafts were drawn from."""
    p = torch.tensor([[0.5, 0.25, 0.25]] * 3)
    q = torch.tensor([[1.0, 0.0, 0.0]] * 3)
    for v, x in ((0.0, 0), (0.49, 0), (0.5, 1), (0.75, 2)):
        v = torch.tensor([v])
        for probs in (q, None):
            # refused as the first draft, and behind an accepted one
            got = run(p, [0, token, 0], [0, 3], torch.zeros(3), v, 2, probs)
            assert got == ([[x, -1, -1]], [[0, -1, -1]], [1])
            got = run(p, [0, 0, token], [0, 3], torch.zeros(3), v, 2, probs)
            assert got == ([[0, x, -1]], [[0, 1, -1]], [2])
        got = run(p, [0, token, token], [0, 3], torch.zeros(3), v, 2, None, [-1, 0, 0])
        assert got == ([[x, -1, -1]], [[0, -1, -1]], [1])
    assert rarn.watchdog() == INDEX_BIT
