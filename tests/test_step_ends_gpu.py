"""GPU tests at the ends of a step's ranges: sequences around 48 KB of shared memory, no
sequences, spoiled pages given back."""
import os
import subprocess
import sys

import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
from test_pages_gpu import check_step, ints, make, same_state

pytestmark = pytest.mark.gpu

INDEX_BIT = 16


@pytest.fixture(autouse=True)
def _watchdog():
    rarn.watchdog(clear=True)
    yield


def test_sequences_whose_sums_just_fit_the_shared_memory_of_any_kernel():
    """In a process of their own: a larger step before would have raised the limit."""
    here = os.path.dirname(os.path.abspath(__file__))
    run = ("import sys; sys.path[:0] = %r; import test_pages_gpu as p\n"
           "for B in (6125, 6126, 6143, 6144): p.test_a_run_of_steps_and_trims(B, 2, 4, 5)"
           % [here, os.path.dirname(here)])
    got = subprocess.run([sys.executable, "-c", run], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr


@pytest.mark.parametrize("tokens", [0, 1, 700])
def test_no_sequences(tokens):
    pages = rarn.KVPages.empty(0, 4, 8, 16)
    none = ints([])
    starts, slots, positions, served = rarn.kv_step(pages, none, none, tokens)
    assert starts.tolist() == [0] and int(served) == 0
    assert slots.tolist() == [-1] * tokens and positions.tolist() == [0] * tokens
    rarn.kv_trim(pages, none)
    assert int(pages.free_count) == 8 and pages.free_pages.tolist() == list(range(7, -1, -1))
    assert rarn.watchdog() == 0


def test_a_spoiled_page_is_given_back_as_it_is():
    """It keeps its place among the free ones: the step that takes it has no slots for its
    tokens, and the pages around it are none the wiser."""
    pages, model = make(2, 4, 8, 4)
    check_step(pages, model, [0, 0], [6, 5], 11)
    for page in (8, -7):
        right = int(pages.page_table[0, 1])
        pages.page_table[0, 1] = page
        rarn.kv_trim(pages, ints([4, 5]))
        assert rarn.watchdog(clear=True) == INDEX_BIT
        n = int(pages.free_count)
        assert n == 5 and int(pages.free_pages[n - 1]) == page
        assert pages.page_table[0].tolist()[1:] == [-1] * 3
        slots, positions = rarn.kv_step(pages, ints([4, 5]), ints([2, 4]), 6)[1:3]
        assert rarn.watchdog(clear=True) == INDEX_BIT
        assert slots.tolist()[:2] == [-1, -1] and min(slots.tolist()[2:]) >= 0
        assert positions.tolist() == [4, 5, 5, 6, 7, 8]
        rarn.kv_trim(pages, ints([6, 5]))
        assert rarn.watchdog(clear=True) == 0
        pages.page_table[0, 1] = right
        same_state(pages, model)
