"""Layer norms of rows longer than 10240 columns, whose gradient kernel holds
one row per block, and dropout of tensors at any address, four elements of a
counter at a time."""
import pytest

import operators_cases as C

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D", [(3, 10248), (200, 12288), (5, 12289), (2, 16384), (170, 16383), (4, 16392), (3, 20480), (2, 20488)])
@pytest.mark.parametrize("type_", ["bf16", "fp16", "fp32"])
def test_norm_wide_rows(T, D, type_):
    C.norm_forward_case(T, D, type_, seed=T + D)
    C.norm_backward_case(T, D, type_, seed=T + D)


@pytest.mark.parametrize("shape", [(1, 1), (1, 3), (1, 4), (1, 5), (130, 1001), (3, 70001)])
@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("type_", ["bf16", "fp16", "fp32"])
def test_dropout_unaligned(shape, offset, type_):
    C.dropout_case(shape, type_, 0.3, seed=sum(shape) + offset, offset=offset)
