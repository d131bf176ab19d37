"""The bounds-checked build of the operators over long runs of one id, every
number of merges, and operands that lie between each other's rows, in a child
process that loads it first (tests/checked_operators_more_run.py)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_no_out_of_range_access():
    run = subprocess.run([sys.executable, os.path.join(HERE, "checked_operators_more_run.py")], capture_output=True,
                         text=True, timeout=1800)
    assert run.returncode == 0, f"{run.stdout[-3000:]}\n{run.stderr[-3000:]}"
    assert "checked operators ok" in run.stdout
