"""Child process of tests/test_checked_matrix_gpu.py (not a test module).

Builds the bounds-checked library (-DMHCPB_CHECKED) beside the product one,
loads it before anything else, runs the feed-forward block and the orthogonalised
update over the shapes where their accesses could go wrong, and checks that no
kernel found an access outside its buffer and that the results still match the
oracle.  Exits non-zero on any failure."""
import os
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

from rms_backward_gb300 import abi  # noqa: E402
from rms_backward_gb300 import build as B  # noqa: E402

LIB = B.build(extra_flags=["-DMHCPB_CHECKED"], out_dir=os.path.join(B.BUILD, "checked"))
abi.load(LIB)

import torch  # noqa: E402

import matrix_cases as M  # noqa: E402


def no_sites(label):
    torch.cuda.synchronize()
    checked, sites = abi.mhcpb_debug_checked_matrix_sites()
    assert checked, "the loaded library is not a checked build"
    bad = {k: v for k, v in sites.items() if v}
    assert not bad, f"{label}: out-of-range accesses (family: 1 + site) {bad}"


def feed_forward():
    for T, D, F in ((1, 1, 1), (1, 8, 8), (2, 7, 3), (3, 75, 141), (4, 1001, 77), (1, 2048, 136), (5, 100, 136), (127, 129, 131),
                    (128, 128, 128), (129, 320, 257), (300, 65, 700), (600, 1048, 2056), (700, 1033, 3431)):
        for type_, act in (("bf16", "silu"), ("fp16", "gelu")):
            M.ffn_forward_case(T, D, F, type_, act, seed=T)
            M.ffn_forward_case(T, D, F, type_, act, train=False, seed=T)
            M.ffn_backward_case(T, D, F, type_, act, seed=T)
            M.ffn_backward_case(T, D, F, type_, act, grad_type="fp32", accumulate=True, seed=T)
            no_sites(f"T={T} D={D} F={F} {type_}")
    for pad in (8, 64):
        M.ffn_forward_case(40, 72, 200, "bf16", pad=pad)
        M.ffn_forward_case(2, 72, 200, "bf16", pad=pad)
        M.ffn_backward_case(40, 72, 200, "bf16", pad=pad)
        no_sites(f"pad={pad}")


def orthogonalise():
    for mm, n in ((1, 1), (1, 20), (9, 1), (17, 5), (24, 2048), (2048, 24), (32, 700), (33, 40), (64, 200), (100, 100), (127, 129),
                  (257, 130), (300, 1001), (2300, 2310), (2600, 2305)):
        for type_ in ("fp32", "bf16"):
            M.orthogonalize_case(mm, n, type_, seed=mm)
            no_sites(f"{mm} x {n} {type_}")
    for mm, n in ((40, 72), (72, 40), (20, 72), (400, 520)):
        M.orthogonalize_case(mm, n, "fp32", pad=8)
        M.orthogonalize_case(mm, n, "fp16", pad=64)
        no_sites(f"{mm} x {n} with gaps")


if __name__ == "__main__":
    for step in (feed_forward, orthogonalise):
        step()
        print(f"{step.__name__}: no out-of-range access, parity holds", flush=True)
    print("checked matrix operators ok")
