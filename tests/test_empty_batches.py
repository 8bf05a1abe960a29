"""Calls without rows or sequences: addresses of empty tensors are null, and nothing is
read from them."""
import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
import test_block_host as block
import test_pages_host as pages
from test_block_host import INVALID, OK, lib  # noqa: F401  (the fixture)


@pytest.mark.parametrize("gate,want", [
    (dict(n=0), OK), (dict(n=0, data=None), OK), (dict(n=0, data=None, stride=0), OK),
    (dict(n=5, index=None, data=None), OK),
    (dict(n=5, index=1 << 50), OK), (dict(n=0, index=1 << 50), OK), (dict(n=-1), INVALID),
    (dict(n=-1, index=1 << 50), INVALID),
])
def test_no_rows_with_gates(lib, gate, want):  # noqa: F811
    none = rarn.Rows(None, block.H, block.BF16)
    assert block.call(lib, T=0, y=none, h=none, x=none, r=none, gate=block.gate(**gate)) == want


def test_a_gate_without_rows_needs_an_empty_batch(lib):  # noqa: F811
    for index in (None, 1 << 50):
        assert block.call(lib, gate=block.gate(n=0, index=index)) == INVALID


def test_no_sequences_pass_the_checks(lib):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only without a device")
    none = dict(sequences=0, page_table=None, held=None)
    assert pages.step(lib, pages.pages(**none), ctx=None, new=None) == pages.CUDA
    assert pages.trim(lib, pages.pages(**none), None) == OK
    for f in ("page_table", "held"):
        assert pages.step(lib, pages.pages(sequences=1, **{f: None})) == INVALID
    for f in ("free_pages", "free_count", "ticket"):
        assert pages.step(lib, pages.pages(**none, **{f: None})) == INVALID


@pytest.mark.gpu
@pytest.mark.parametrize("gates,index", [(0, False), (0, True), (1, False), (3, True)])
def test_no_rows_through_the_binding(gates, index):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    gm = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    gate = torch.ones(gates, 64, dtype=torch.bfloat16, device="cuda")
    at = torch.empty(0, dtype=torch.int32, device="cuda") if index else None
    y = rarn.gated_add_rms_norm(x, x.clone(), gm, gm, 1e-6, gate=gate, gate_index=at)
    assert y.shape == (0, 64)
