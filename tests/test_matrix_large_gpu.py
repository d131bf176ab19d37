"""Tensors of more than 2^31 elements through the feed-forward block and the
orthogonalised update, where a 32-bit index would wrap."""
import numpy as np
import pytest
import torch

import oracle.mhcm_oracle as O
import rms_backward_gb300 as m

import matrix_cases as M
from matrix_cases import DEV, f64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LIMIT = 1 << 31


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("F", [2560, 2561])
def test_tokens_times_hidden(F):
    """gate, up and the products in the workspace pass 2^31 elements; rows are compared at both ends and
    around elements 2^30 and 2^31, the weights' gradients with tokens that are zero but for those rows."""
    D, T = 40, LIMIT // F + 900
    rows = torch.tensor(sorted({0, 1, T // 3, (1 << 30) // F, LIMIT // F - 1, LIMIT // F, LIMIT // F + 1, T - 2, T - 1}))
    g, xr, wg, wu, wd = M.inputs(len(rows), D, F, BF, 5)
    x, dy = torch.zeros(T, D, dtype=BF, device=DEV), torch.zeros(T, D, dtype=BF, device=DEV)
    dyr = torch.randn(len(rows), D, generator=g).to(BF).to(DEV)
    at = rows.to(DEV)
    x[at], dy[at] = xr, dyr
    y, dx = torch.empty_like(x), torch.empty_like(x)
    gate, up = (torch.empty(T, F, dtype=BF, device=DEV) for _ in range(2))
    ws = torch.empty(m.mhc_ffn_forward_workspace_bytes(T, D, F), dtype=torch.uint8, device=DEV)
    m.mhc_ffn_forward(x, wg, wu, wd, y, ws, gate, up)
    ref, bound = O.ffn_forward(*map(f64, (xr, wg, wu, wd)), "silu", "bf16")
    for name, t, r, b in zip(("y", "gate", "up"), (y, gate, up), ref, bound):
        M.within(name, t[at], r, b)
        assert torch.count_nonzero(t.any(1)) <= len(rows)
    del ws
    ws = torch.empty(m.mhc_ffn_backward_workspace_bytes(T, D, F), dtype=torch.uint8, device=DEV)
    grads = [torch.empty(w.shape, device=DEV) for w in (wg, wu, wd)]
    m.mhc_ffn_backward(x, wg, wu, wd, gate, up, dy, dx, *grads, ws)
    ref, bound = O.ffn_backward(*map(f64, (xr, wg, wu, wd, gate[at], up[at], dyr)), "silu", "bf16", "fp32")
    for name, t, r, b in zip(("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down"), (dx[at], *grads), ref, bound):
        M.within(name, t, r, b)


def test_weights():
    """Weights of 2^31 elements and more, one token (its own kernels) and a few."""
    D, F = 49160, 43696
    assert D * F > LIMIT
    wg, wu = (torch.zeros(F, D, dtype=BF, device=DEV) for _ in range(2))
    wd = torch.zeros(D, F, dtype=BF, device=DEV)
    # a few weights in the first and last rows: act(g) u = 64 * 2 in every hidden place that they reach
    wg[0, :4], wu[0, :2] = 16.0, 1.0
    wg[F - 1, D - 4:], wu[F - 1, D - 2:] = 16.0, 1.0
    wd[0, 0], wd[D - 1, F - 1], wd[D - 1, 0] = 1.0, 2.0, -1.0
    for T in (1, 6):
        x = torch.ones(T, D, dtype=BF, device=DEV)
        y = torch.empty_like(x)
        ws = torch.empty(m.mhc_ffn_forward_workspace_bytes(T, D, F), dtype=torch.uint8, device=DEV)
        m.mhc_ffn_forward(x, wg, wu, wd, y, ws)
        want = torch.zeros_like(x)
        want[:, 0], want[:, D - 1] = 128.0, 128.0
        assert torch.equal(y, want)


@pytest.mark.parametrize("tall", [False, True])
def test_orthogonalise(tall):
    """Rows with disjoint supports are the singular vectors: out is each row times f(s) / s."""
    s, l = 2056, (1 << 20)
    assert s * l > LIMIT
    g = torch.zeros(s, l, dtype=BF, device=DEV)
    cols = torch.arange(l, device=DEV)
    size = torch.exp2((torch.arange(s, device=DEV) % 4).float())          # rows of four sizes
    g[cols % s, cols] = size[cols % s].to(BF)
    norms = g.float().square().sum(1).sqrt().double().cpu().numpy()
    v = norms / np.sqrt((norms ** 2).sum())
    f = v.copy()
    for _ in range(5):
        f = O.A * f + O.B * f ** 3 + O.C * f ** 5
    if tall:
        g = g.t().contiguous()
    out = torch.empty_like(g)
    ws = torch.empty(m.mhc_orthogonalize_workspace_bytes(*g.shape), dtype=torch.uint8, device=DEV)
    m.mhc_orthogonalize(g, out, ws)
    del ws
    if tall:
        out = out.t()
    got = out[cols % s, cols].double().cpu().numpy()
    row = (np.arange(l) % s)
    want = (size.double().cpu().numpy() * f / norms)[row]
    # one direction a row: X's copy and B's diagonal are rounded to 2^-11 in each of five steps, B X is at
    # most 2.81 X, a step changes a relative error by a factor of at most |s f'(s) / f(s)| < 4, and most
    # by less than 1 once s is large; the output's rounding adds 2^-8
    assert np.all(np.abs(got - want) <= np.abs(want) * (2.0 ** -8 + 16 * 2.0 ** -11))
    assert torch.count_nonzero(out[0]) == torch.count_nonzero(g.t()[0] if tall else g[0])
