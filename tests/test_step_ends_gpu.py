"""GPU tests at the ends of a step's ranges."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_sequences_whose_sums_just_fit_the_shared_memory_of_any_kernel():
    """In a process of their own: a larger step before would have raised the limit."""
    here = os.path.dirname(os.path.abspath(__file__))
    run = ("import sys; sys.path[:0] = %r; import test_pages_gpu as p\n"
           "for B in (6125, 6126, 6143, 6144): p.test_a_run_of_steps_and_trims(B, 2, 4, 5)"
           % [here, os.path.dirname(here)])
    got = subprocess.run([sys.executable, "-c", run], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stderr
