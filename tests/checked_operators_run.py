"""Child process of tests/test_checked_operators_gpu.py (not a test module).

Builds the bounds-checked library (-DMHCPB_CHECKED) beside the product one,
loads it before anything else, runs the operators around the stage over the
shapes where their accesses could go wrong, and checks that no kernel found
an access outside its buffer and that the results still match the oracle.
Exits non-zero on any failure."""
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

import operators_cases as C  # noqa: E402


def no_sites(label):
    torch.cuda.synchronize()
    checked, sites = abi.mhcpb_debug_checked_operator_sites()
    assert checked, "the loaded library is not a checked build"
    bad = {k: v for k, v in sites.items() if v}
    assert not bad, f"{label}: out-of-range accesses (family: 1 + site) {bad}"


def embedding():
    for T, V, D, n in ((1, 1, 1, 1), (3, 50, 5120, 4), (77, 9, 1285, 4), (40, 300, 40, 16), (0, 5, 8, 2)):
        for type_, wide in (("bf16", True), ("fp32", False)):
            C.embed_forward_case(T, V, D, n, type_, wide, seed=T + D)
            C.embed_forward_case(T, V, D, n, type_, wide, seed=T + D, offset=1)
            no_sites(f"embed_forward T={T} V={V} D={D} n={n} {type_}")
    for T, V, D, n in ((1, 1, 1, 1), (1, 70, 8, 4), (33, 5, 1285, 1), (500, 2000, 40, 4), (4096, 37, 16, 2),
                       (4097, 5000, 8, 1), (9001, 64, 3, 4), (300000, 5000, 1, 1), (0, 5, 8, 2)):
        for accumulate in (False, True):
            C.embed_backward_case(T, V, D, n, True, accumulate, seed=T + D)
            C.embed_backward_case(T, V, D, n, False, accumulate, seed=T + D, skew=True, offset=1)
            no_sites(f"embed_backward T={T} V={V} D={D} n={n} accumulate={accumulate}")


def norms():
    for T, D in ((1, 1), (1, 5120), (3, 2), (5, 7), (33, 40), (300, 128), (17, 1285), (9, 8200), (2, 20000), (3, 70001),
                 (700, 64), (2, 131072), (400, 5120), (200, 10240), (160, 12288), (3, 16383), (2, 16384)):
        for type_ in ("bf16", "fp32"):
            C.norm_forward_case(T, D, type_, seed=T + D)
            C.norm_backward_case(T, D, type_, seed=T + D)
            no_sites(f"norm T={T} D={D} {type_}")
    for D, pad in ((40, 8), (40, 1), (1285, 3)):
        C.norm_forward_case(200, D, "bf16", seed=D, pad=pad)
        C.norm_backward_case(200, D, "bf16", seed=D, pad=pad)
        no_sites(f"norm strides D={D} pad={pad}")


def streams():
    for T, D in ((1, 1), (1, 5120), (2, 3), (5, 8), (33, 41), (70, 320), (9, 1285), (3, 8200), (2, 33000), (400, 72),
                 (400, 5120), (161, 8192), (155, 4097)):
        C.collapse_case(T, D, seed=T + D)
        no_sites(f"collapse T={T} D={D}")
        C.update_case(T, D, 0.0, seed=T + D)
        no_sites(f"update T={T} D={D}")
    for T, D in ((7, 40), (5, 1285)):
        C.update_case(T, D, 0.3, seed=T)
        C.update_case(T, D, 0.3, seed=T, in_place=True)
        C.collapse_case(T, D, seed=T, residual=False, params=False)
        no_sites(f"update with dropout T={T} D={D}")
    for shape, offset in (((1, 1), 0), ((3, 5), 0), ((64, 40), 0), ((7, 1285), 1), ((130, 1001), 3)):
        for type_ in ("bf16", "fp32"):
            C.dropout_case(shape, type_, 0.25, seed=1, offset=offset)
            no_sites(f"dropout {shape} {type_}")


if __name__ == "__main__":
    for step in (embedding, norms, streams):
        step()
        print(f"{step.__name__}: no out-of-range access, parity holds", flush=True)
    print("checked operators ok")
