"""GPU tests at the ends of a step's ranges: sequences around 48 KB of shared memory,
no sequences."""
import os
import subprocess
import sys

import pytest
import torch

import residual_add_rmsnorm_gb300 as rarn
from test_pages_gpu import ints

pytestmark = pytest.mark.gpu


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
