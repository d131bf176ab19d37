"""Up to 64 tokens a, dg and du are kept as two 16-bit numbers: what their sum does
where single numbers would not, or would do better."""
import numpy as np
import pytest
import torch

import oracle.mhcm_oracle as O
import rms_backward_gb300 as m

import matrix_cases as M
from matrix_cases import DEV, f64

pytestmark = pytest.mark.gpu
INF = float("inf")


def _silu(g):
    q = 1.0 / (1.0 + np.exp(-g))
    return g * q, q * (1.0 + g * (1.0 - q))


@pytest.mark.parametrize("type_", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 4, 5, 33, 40, 64, 65, 130])
@pytest.mark.parametrize("D,F", [(72, 264), (75, 141), (520, 3000)])
def test_infinite_weights(T, D, F, type_):
    """An infinite weight makes the outputs that it reaches what the formula says: infinite with the sign of
    what it is multiplied by (none of which is zero here), NaN where two of opposite signs meet; the
    others keep their bits."""
    dtype = M.TYPES[type_]
    g, x, wg, wu, wd = M.inputs(T, D, F, dtype, T + D)
    gate, up = (M.put(0.5 + torch.rand(T, F, generator=g), dtype) for _ in range(2))
    up *= torch.where(torch.rand(T, F, generator=g) < 0.5, -1.0, 1.0).to(dtype).to(DEV)
    dy = M.put(torch.randn(T, D, generator=g), dtype)
    ws, _ = M.scratch(max(m.mhc_ffn_forward_workspace_bytes(T, D, F), m.mhc_ffn_backward_workspace_bytes(T, D, F)))

    def run(wg_, wu_, wd_):
        y, dx = torch.empty_like(x), torch.empty_like(x)
        m.mhc_ffn_forward(x, wg, wu, wd_, y, ws)
        m.mhc_ffn_backward(x, wg_, wu_, wd, gate, up, dy, dx, None, None, None, ws)
        return y, dx

    clean = run(wg, wu, wd)
    bg, bu, bd = wg.clone(), wu.clone(), wd.clone()
    bd[1, 3], bd[D // 2, F - 1], bd[D - 1, 5], bd[D - 1, F // 2] = INF, -INF, INF, INF
    bg[3, 2], bg[F // 2, D - 2], bu[0, 0], bu[F - 1, D - 2] = INF, -INF, INF, INF
    got = run(bg, bu, bd)
    with np.errstate(invalid="ignore"):
        a = _silu(f64(x) @ f64(wg).T)[0] * (f64(x) @ f64(wu).T)
        act, slope = _silu(f64(gate))
        da = f64(dy) @ f64(wd)
        dg, du = da * f64(up) * slope, da * act
        assert all(abs(v[:, cols]).min() > 0 for v, cols in ((a, [3, F - 1, 5, F // 2]), (dg, [3, F // 2]), (du, [0, F - 1])))
        want = [a @ f64(bd).T, dg @ f64(bg) + du @ f64(bu)]
    reached = [[1, D // 2, D - 1], [0, 2, D - 2]]
    for name, w, q, c, cols in zip(("y", "grad_x"), want, got, clean, reached):
        keep = [i for i in range(D) if i not in cols]
        assert torch.equal(q[:, keep], c[:, keep]), name
        assert not np.isfinite(w[:, cols]).any() and np.isfinite(w[:, keep]).all()
        assert np.array_equal(f64(q[:, cols]), w[:, cols], equal_nan=True), name


@pytest.mark.parametrize("type_", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 4, 5, 33, 64])
@pytest.mark.parametrize("D,F", [(72, 264), (75, 141)])
def test_small_values_lose_nothing(T, D, F, type_):
    """a, dg and du of some 2^-18, of which FP16 alone keeps seven bits: y's and grad_x's only rounding to 16
    bits is the output's.  (What is kept of them beside the first number has steps of 2^-36 in FP16, 16 bits in
    BF16; with FP32 sums that is below 2^-13 of the result in the 2-norm.)"""
    dtype = M.TYPES[type_]
    g, x, wg, wu, wd = M.inputs(T, D, F, dtype, T + F)
    small, large = 2.0 ** -8, 2.0 ** 8      # (powers of two: the weights stay as they are but for their size)
    gate, up = (M.put(torch.randn(T, F, generator=g), dtype) for _ in range(2))
    dy = M.put(2.0 ** -14 * torch.randn(T, D, generator=g), dtype)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    ws, _ = M.scratch(max(m.mhc_ffn_forward_workspace_bytes(T, D, F), m.mhc_ffn_backward_workspace_bytes(T, D, F)))
    forward, backward = (x, wg * small, wu * small, wd * large), (x, wg * large, wu * large, wd * 2.0 ** -4)
    m.mhc_ffn_forward(*forward, y, ws)
    m.mhc_ffn_backward(*backward, gate, up, dy, dx, None, None, None, ws)
    ref = [O.ffn_forward(*map(f64, forward), "silu", type_)[0][0],
           O.ffn_backward(*map(f64, (*backward, gate, up, dy)), "silu", type_, type_)[0][0]]
    norm = lambda v: (v ** 2).sum() ** 0.5  # noqa: E731
    for name, got, r in zip(("y", "grad_x"), (y, dx), ref):
        once = torch.from_numpy(r).to(dtype).double().numpy()
        assert norm(f64(got) - r) <= norm(once - r) + 2.0 ** -13 * norm(r), name
