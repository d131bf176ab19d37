"""Norm gradients of rows that lie far from zero, whose mean is hundreds of
times their deviation.  z = (u - mean) rstd has one rounding of a difference
and one of a product, so with u exact (a plain row; a collapsed one whose gates
are powers of two and whose streams are small integers) its error is two units
of 2^-24 of |z| itself, not of |mean| rstd: the bounds below are
oracle/mhcs_oracle.py's with |u - mean| in the place of |u| + |mean|.

Chains: rows as in operators_cases.py.  A row's term of a parameter gradient is
two roundings of z and one product from exact, and passes through the additions of its
group's rows (at least 152 groups), of a block's groups (at most 15), and of the
parts: at most 19 by a thread, then 16; 64 + T / 152 covers them."""
import numpy as np
import pytest
import torch

import oracle.mhcs_oracle as S
import rms_backward_gb300 as m

import operators_cases as C
from operators_cases import DEV, DTYPES, check, empty, gen, normal, np64, scratch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _statistics(u):
    _, mean, rstd, *_ = S.norm_forward(u, 1.0, 0.0, 1e-5)
    return (torch.from_numpy(a).float() for a in (mean, rstd))


def _reference(u, gy, gamma, mean, rstd):
    """(du, dgamma, dbeta) and their magnitudes about the row's mean."""
    ref, _ = S.norm_backward(u, gy, gamma, mean, rstd)
    z, w = np.abs(u - mean[:, None]) * rstd[:, None], np.abs(gy * gamma)
    du = rstd[:, None] * (w + w.mean(1, keepdims=True) + z * (w * z).mean(1, keepdims=True))
    return ref, (du, (np.abs(gy) * z).sum(0), np.abs(gy).sum(0))


def _check_parameters(T, got, ref, mag):
    for k, name in enumerate(("grad_gamma", "grad_beta")):
        check(name, got[k], ref[1 + k], mag[1 + k], 64 + -(-T // 152))


# one, two and four vectors a thread, aligned and not, and rows that are read again
WIDTHS = [40, 1280, 1285, 5120, 12288, 12289, 20488]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("T", [3, 400])
@pytest.mark.parametrize("type_,offset", [("fp32", 1000.0), ("fp16", 300.0), ("bf16", 300.0)])
def test_norm_gradient(T, D, type_, offset):
    g = gen(T + D)
    dt = DTYPES[type_]
    x, gy, gamma = (offset + normal(g, T, D)).to(dt), normal(g, T, D, dtype=dt), normal(g, D)
    mean, rstd = _statistics(np64(x))
    gx, grads = empty(T, D, dtype=dt), (empty(D), empty(D))
    m.mhc_layernorm_backward(x.to(DEV), gy.to(DEV), gamma.to(DEV), mean.to(DEV), rstd.to(DEV), gx, *grads,
                             scratch(m.mhc_layernorm_workspace_bytes(T, D)))
    ref, mag = _reference(np64(x), np64(gy), np64(gamma), np64(mean), np64(rstd))
    _check_parameters(T, grads, ref, mag)
    check("grad_x", gx, ref[0], mag[0], 2 * C.row_chain(D), type_)


@pytest.mark.parametrize("D", [40, 1280, 1285, 5120, 8192, 8200, 5121, 10248])
@pytest.mark.parametrize("T", [3, 400])
def test_collapse_gradient(T, D):
    """u = X_0 + X_1 / 2 + X_2 / 4 + 2 X_3, about 300, is exact in FP32."""
    g = gen(T + D)
    x = torch.full((T, 4 * D), 80.0)
    x[:, :D] += torch.randint(-2, 3, (T, D), generator=g)
    h = C.gates(g, T)
    h[:, :4] = torch.tensor([1.0, 0.5, 0.25, 2.0])
    x, gy, gamma = x.to(BF), normal(g, T, D, dtype=BF), normal(g, D)
    u, _ = S.collapse(np64(x), np64(h))
    mean, rstd = _statistics(u)
    gx, gh, grads = empty(T, 4 * D, dtype=BF), empty(T, 24), (empty(D), empty(D))
    m.mhc_collapse_norm_backward(x.to(DEV), h.to(DEV), gy.to(DEV), gamma.to(DEV), mean.to(DEV), rstd.to(DEV), gx, gh,
                                 *grads, scratch(m.mhc_collapse_norm_workspace_bytes(T, D)))
    ref, mag = _reference(u, np64(gy), np64(gamma), np64(mean), np64(rstd))
    _check_parameters(T, grads, ref, mag)
    pre, xs = np64(h)[:, :4, None], np64(x).reshape(T, 4, D)
    check("grad_x", gx, (pre * ref[0][:, None]).reshape(T, -1), (pre * mag[0][:, None]).reshape(T, -1),
          2 * C.row_chain(D), "bf16")
    check("grad_h", gh[:, :4], (xs * ref[0][:, None]).sum(2), (np.abs(xs) * mag[0][:, None]).sum(2), 2 * C.row_chain(D))


# threads past the row's end in a group of 32, in all their vectors or in some
@pytest.mark.parametrize("D", [1, 40, 41, 64, 1280, 1285, 5128, 12296])
@pytest.mark.parametrize("T", [1, 200])
@pytest.mark.parametrize("type_", ["fp32", "bf16"])
def test_constant_rows_of_large_numbers(T, D, type_):
    """Each row is 2^120 throughout, so z = 0 and du = rstd (w - mean w) are
    finite although mean rstd is not: what lies past a row's end adds nothing.
    (The first gate's gradient is not looked at: its terms, 2^120 du, pass FP32.)"""
    g, dt = gen(T + D), DTYPES[type_]
    x, gy, gamma = torch.full((T, D), 2.0**120, dtype=dt), normal(g, T, D, dtype=dt), normal(g, D)
    mean, rstd = torch.full((T,), 2.0**120), torch.full((T,), 1e-5).rsqrt()
    ref, mag = _reference(np64(x), np64(gy), np64(gamma), np64(mean), np64(rstd))
    gx, grads = empty(T, D, dtype=dt), (empty(D), empty(D))
    m.mhc_layernorm_backward(x.to(DEV), gy.to(DEV), gamma.to(DEV), mean.to(DEV), rstd.to(DEV), gx, *grads,
                             scratch(m.mhc_layernorm_workspace_bytes(T, D)))
    _check_parameters(T, grads, ref, mag)
    assert not grads[0].any()
    check("grad_x", gx, ref[0], mag[0], 2 * C.row_chain(D), type_)
    if type_ != "bf16" or 4 * D > 40000:
        return
    h = torch.zeros(T, 24)
    h[:, 0] = 1.0   # u = X_0
    xs, gh, gx = torch.zeros(T, 4 * D, dtype=BF), empty(T, 24), empty(T, 4 * D, dtype=BF)
    xs[:, :D] = x
    m.mhc_collapse_norm_backward(xs.to(DEV), h.to(DEV), gy.to(DEV), gamma.to(DEV), mean.to(DEV), rstd.to(DEV), gx, gh,
                                 *grads, scratch(m.mhc_collapse_norm_workspace_bytes(T, D)))
    _check_parameters(T, grads, ref, mag)
    assert not grads[0].any() and not gx[:, D:].any() and not gh[:, 1:4].any()
    check("grad_x", gx[:, :D], ref[0], mag[0], 2 * C.row_chain(D), "bf16")
