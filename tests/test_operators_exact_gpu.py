"""Embedding gradients of whole numbers, equal to the last bit, where a run of
one id crosses many chunks, more of them than the joining kernel counts at
once (512), and where ordering takes every number of merges up to four."""
import pytest
import torch

import rms_backward_gb300 as m

import operators_exact as X
from operators_cases import DEV, empty, off_by, scratch

pytestmark = pytest.mark.gpu


def run(T, V, D, n, seed, frequent=0.0, pad=0.0, start=False, offset=0, wide=True):
    ids, grad_x, table, want = X.case(T, V, D, n, seed, frequent, pad, start)
    out = off_by(table if start else empty(V, D), offset)
    ids = ids.to(torch.int64 if wide else torch.int32)
    m.mhc_embed_backward(off_by(ids, offset), off_by(grad_x, 3 * offset), out,
                         scratch(m.mhc_embed_workspace_bytes(T, V, D)), accumulate=start)
    assert X.equal(out, want)


@pytest.mark.parametrize("T,V,D,n", [(200, 3, 24, 4), (5000, 401, 17, 4), (17000, 3, 1032, 4), (40000, 64, 8, 4),
                                     (40000, 64, 9, 1), (70000, 64, 16, 1), (131073, 5, 3, 2)])
@pytest.mark.parametrize("frequent", [0.8, 1.0])
@pytest.mark.parametrize("start,offset", [(False, 0), (True, 1)])
def test_long_runs(T, V, D, n, frequent, start, offset):
    run(T, V, D, n, seed=T + D, frequent=frequent, pad=0.01, start=start, offset=offset, wide=not start)


# one tile; one, two, three and four merges, the last run of each short
@pytest.mark.parametrize("T", [1, 4, 5, 1024, 4095, 4096, 4097, 16384, 16385, 16500, 262144, 262145, 4194304, 4194400])
@pytest.mark.parametrize("V,frequent", [(70001, 0.0), (70001, 0.5)])
def test_every_number_of_merges(T, V, frequent):
    run(T, V, 1, 1, seed=T, frequent=frequent, pad=0.02)
