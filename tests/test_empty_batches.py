"""Calls without sequences: addresses of empty tensors are null, and nothing is read from
them."""
import pytest
import torch

import test_pages_host as pages
from test_pages_host import INVALID, OK, lib  # noqa: F401  (the fixture)


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
