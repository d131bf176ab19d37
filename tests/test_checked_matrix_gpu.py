"""The bounds-checked build of the feed-forward block and the orthogonalised update
(include/mhcpb.h, mhcpb_debug_checked_matrix_sites): in a child process that
loads it first (tests/checked_matrix_run.py), no access falls outside its buffer."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_no_out_of_range_access():
    run = subprocess.run([sys.executable, os.path.join(HERE, "checked_matrix_run.py")], capture_output=True, text=True,
                         timeout=1800)
    assert run.returncode == 0, f"{run.stdout[-3000:]}\n{run.stderr[-3000:]}"
    assert "checked matrix operators ok" in run.stdout
