"""The bounds-checked build of the operators around the stage (include/mhcpb.h,
mhcpb_debug_checked_operator_sites): in a child process that loads it first
(tests/checked_operators_run.py), no access falls outside its buffer, and the
results still match the oracle."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_checked_operators_find_no_out_of_range_access():
    run = subprocess.run([sys.executable, os.path.join(HERE, "checked_operators_run.py")], capture_output=True,
                         text=True, timeout=1800)
    assert run.returncode == 0, f"{run.stdout[-3000:]}\n{run.stderr[-3000:]}"
    assert "checked operators ok" in run.stdout
