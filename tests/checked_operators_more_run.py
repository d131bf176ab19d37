"""Child process of tests/test_checked_operators_more_gpu.py (not a test module).

Runs, in the bounds-checked build (made as by tests/checked_operators_run.py, or
taken if it is newer than its sources), the embedding gradient over long runs
and every number of merges, and norms of column slices of one buffer.  Exits
non-zero when a kernel found an access outside its buffer or a result is
wrong."""
import glob
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

from rms_backward_gb300 import abi  # noqa: E402
from rms_backward_gb300 import build as B  # noqa: E402

DIR = os.path.join(B.BUILD, "checked")
LIB = os.path.join(DIR, os.path.basename(B.LIB))
SOURCES = [f for d in (B.CSRC, B.INCLUDE) for f in glob.glob(os.path.join(d, "*"))]
if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(map(os.path.getmtime, SOURCES)):
    LIB = B.build(extra_flags=["-DMHCPB_CHECKED"], out_dir=DIR)
abi.load(LIB)

import torch  # noqa: E402

import test_operators_exact_gpu as E  # noqa: E402
import test_operators_slices_gpu as L  # noqa: E402


def no_sites(label):
    torch.cuda.synchronize()
    checked, sites = abi.mhcpb_debug_checked_operator_sites()
    assert checked, "the loaded library is not a checked build"
    bad = {k: v for k, v in sites.items() if v}
    assert not bad, f"{label}: out-of-range accesses (family: 1 + site) {bad}"


if __name__ == "__main__":
    for T, V, D, n in ((200, 3, 24, 4), (5000, 401, 17, 4), (40000, 64, 8, 4), (40000, 64, 9, 1)):
        for start in (False, True):
            E.run(T, V, D, n, seed=T, frequent=0.8, pad=0.01, start=start, offset=int(start))
            no_sites(f"embed_backward T={T} V={V} D={D} n={n} start={start}")
    for T in (5, 4096, 4097, 16500, 262145, 4194400):
        E.run(T, 70001, 1, 1, seed=T, frequent=0.5, pad=0.02)
        no_sites(f"embed_backward T={T}")
    for T, D, gap in ((5, 7, 0), (5, 64, 7), (700, 1285, 0), (700, 1285, 1), (700, 1280, 8), (400, 5120, 7), (2, 20481, 0),
                      (200, 12289, 1)):
        for type_ in ("bf16", "fp32"):
            L.test_norm_in_slices_of_one_buffer(T, D, gap, type_)
            no_sites(f"norm in slices T={T} D={D} gap={gap} {type_}")
    print("checked operators ok")
