"""Norms of rows at any address in every type and for every number of warps a
row can have, and forwards of rows far from zero in each of the kernels (rows
in registers, through shared memory, read again)."""
import numpy as np
import pytest
import torch

import oracle.mhcs_oracle as S
import rms_backward_gb300 as m

import operators_cases as C
from operators_cases import DEV, DTYPES, check, empty, gen, normal, np64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("D", [9, 33, 255, 1281, 2561, 4097, 5119, 8193, 10241, 12289, 13313, 16383, 18431])
@pytest.mark.parametrize("type_", ["bf16", "fp16", "fp32"])
def test_group_shapes_in_every_type(D, type_):
    T = max(320, min(2400, 3_000_000 // D))   # above two rows per SM, the forward goes through shared memory
    C.norm_forward_case(T, D, type_, seed=D)
    C.norm_backward_case(T, D, type_, seed=D)


def _statistics_hold(u, mean, rstd, D):
    """A mean of `offset` and a deviation of 1.  Any mean the kernels form (a
    thread's, a warp's or the row's) is off by at most d = (64 + D / 256) 2^-24
    offset: a thread adds up at most 32 values, or D / 256 of rows that are read
    again, and two times 32 lanes or warps are joined in five steps.  About means that are off by d, the sum of squares changes by
    D d^2, and the warps' share of it by twice d times their distance, below 1:
    2 d + d^2 of the variance, half of that of rstd; and the sums' own
    rounding.  (A mean of squares less the square of the mean would be off by
    2^-24 offset^2 and more.)"""
    _, want_mean, want, *_ = S.norm_forward(u, 1.0, 0.0, 1e-5)
    dev = 1.0 / want
    d = (64 + D / 256) * 2.0**-24 * np.abs(want_mean) / dev
    assert np.all(np.abs(np64(mean) - want_mean) <= d * dev)
    assert np.all(np.abs(np64(rstd) / want - 1) <= d + d * d + C.row_chain(D) * 2.0**-24)


@pytest.mark.parametrize("T,D", [(7, 515), (7, 520), (700, 1280), (700, 1285), (700, 5120), (700, 5121), (320, 10240),
                                 (320, 16384), (3, 20488), (3, 20481)])
@pytest.mark.parametrize("type_,offset", [("fp32", 1000.0), ("fp16", 300.0), ("bf16", 300.0)])
def test_forward_far_from_zero(T, D, type_, offset):
    x = (offset + normal(gen(T + D), T, D)).to(DTYPES[type_])
    y, mean, rstd = empty(T, D, dtype=x.dtype), empty(T), empty(T)
    m.mhc_layernorm_forward(x.to(DEV), None, None, y, mean, rstd)
    _statistics_hold(np64(x), mean, rstd, D)
    # from the kernel's own statistics: a difference and a product, then y's own rounding
    z = (np64(x) - np64(mean)[:, None]) * np64(rstd)[:, None]
    check("y", y, z, np.abs(z), 4, type_)


@pytest.mark.parametrize("T,D", [(7, 520), (700, 1280), (700, 1285), (700, 5120), (700, 5121), (320, 8192), (3, 10248), (3, 10249)])
def test_collapse_far_from_zero(T, D):
    """u = X_0 + X_1 / 2 + X_2 / 4 + 2 X_3, about 300, is exact in FP32."""
    g = gen(T + D)
    x = torch.full((T, 4 * D), 80.0)
    x[:, :D] += torch.randint(-2, 3, (T, D), generator=g)
    h = C.gates(g, T)
    h[:, :4] = torch.tensor([1.0, 0.5, 0.25, 2.0])
    u, _ = S.collapse(np64(x), np64(h))
    y, mean, rstd = empty(T, D, dtype=BF), empty(T), empty(T)
    m.mhc_collapse_norm_forward(x.to(BF).to(DEV), h.to(DEV), None, None, y, mean, rstd)
    _statistics_hold(u, mean, rstd, D)
