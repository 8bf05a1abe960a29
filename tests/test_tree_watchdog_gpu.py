"""Failure detection in the attention's kernels without a GPU fault: the test
hook leaves one fill of CTA 0 without some of its bytes, the waits on it run out
within a short limit, the call returns with watchdog bit 5 set, and the join
takes nothing from a segment that was given up."""
import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
from test_tree_gpu import Case

pytestmark = pytest.mark.gpu

WAIT_BIT = 32


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


# two segments of many tiles, spread over all CTAs: CTA 0 begins the first
@pytest.mark.parametrize("n,D,dt", [(20, 128, "bf16"), (20, 64, "f16"), (80, 128, "f16"),
                                    (80, 64, "bf16")])
@pytest.mark.parametrize("fill,left", [(0, 0x01), (5, 0xff), (8, 0x01)])
def test_a_wait_in_the_tiles_runs_out(n, D, dt, fill, left):
    c = Case([150 * 128 * 8], [n], 4, 2, D, dt=dt, page=128, seed=40, mask="chain")
    assert rarn.plan_tree_attention(n, 1, 4, 2, D, 128).startswith("tree.tiles")
    # what earlier calls may have left in the workspace
    ws = torch.full((rarn.tree_attention_workspace_bytes(n, 1, 4, 2, D),), left,
                    dtype=torch.uint8, device="cuda")
    out = torch.full(c.q.shape, -7.0, dtype=c.dt, device="cuda")
    good = c.run()
    torch.cuda.synchronize()
    assert rarn.library().rarn_test_stall(fill, 20_000_000) == 0      # 20 ms
    c.run(out=out, workspace=ws)
    torch.cuda.synchronize()
    assert rarn.watchdog(clear=True) == WAIT_BIT
    # the first key head's segment began in CTA 0: its rows are as they were; the other's
    # are whole
    assert (out[:, :2] == -7.0).all()
    assert torch.equal(out[:, 2:], good[:, 2:])
    # the next call is right, in the same workspace
    c.run(out=out, workspace=ws)
    assert torch.equal(out, good)
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("n,D", [(20, 128), (80, 64)])
def test_a_segment_that_began_elsewhere(n, D):
    """Many sequences: those that CTA 0 finished before its wait ran out are
    whole, those after it as they were or NaN, and no other row is touched."""
    B = 600
    c = Case([300 + i % 50 for i in range(B)], [n] * B, 4, 1, D, page=16, seed=41, mask="chain")
    good = c.run()
    torch.cuda.synchronize()
    ws = torch.full((rarn.tree_attention_workspace_bytes(n * B, B, 4, 1, D),), 0x01,
                    dtype=torch.uint8, device="cuda")
    out = torch.full(c.q.shape, -7.0, dtype=c.dt, device="cuda")
    assert rarn.library().rarn_test_stall(12, 20_000_000) == 0
    c.run(out=out, workspace=ws)
    torch.cuda.synchronize()
    assert rarn.watchdog(clear=True) == WAIT_BIT
    same, kept, nan = out == good, out == -7.0, torch.isnan(out)
    assert (same | kept | nan).all() and (kept | nan).any()
    # (segments lie on the line in order, and CTA 0 has the first part of it)
    assert same[8 * n:].all()
    assert torch.equal(c.run(out=out, workspace=ws), good)
    assert rarn.watchdog() == 0


@pytest.mark.parametrize("n,D,fill", [(1, 128, 0), (1, 64, 3), (3, 256, 2), (6, 128, 1)])
def test_a_wait_in_the_rows_runs_out(n, D, fill):
    """The rows that miss a warp's keys are NaN, the others whole."""
    B = 1200
    c = Case([150] * B, [n] * B, 2, 1, D, page=16, seed=42, mask="chain")
    assert rarn.plan_tree_attention(n * B, B, 2, 1, D, 16).startswith("tree.rows")
    good = c.run()
    torch.cuda.synchronize()
    out = torch.full(c.q.shape, -7.0, dtype=c.dt, device="cuda")
    assert rarn.library().rarn_test_stall(fill, 20_000_000) == 0
    c.run(out=out)
    torch.cuda.synchronize()
    assert rarn.watchdog(clear=True) == WAIT_BIT
    nan = torch.isnan(out)
    assert nan.any() and ((out == good) | nan).all() and not nan[8 * n:].any()
    assert torch.equal(c.run(out=out), good)
    assert rarn.watchdog() == 0
