"""Products whose sums have tens of thousands of terms and more: they are taken in pieces that are added
rounded, since the tensor cores cut what they add, and a sum of one sign loses some 2^-23 of itself with
every 16 terms (2^20 positive ones in one piece: 6.4e-3, 0.8 of that).  Whole numbers to the last bit in every shape of the kernel that takes
pieces, and sums of one sign at the limits of the sizes."""
import numpy as np
import pytest
import torch

import rms_backward_gb300 as m

import matrix_cases as M
from matrix_cases import DEV, f64

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16
# what a sum of positive terms may lose: 2^-23 for each 16 terms of a piece of 32,768, half of that for a
# rounded addition per piece (at most 64 of them here) and per block of a cluster
SUM = 2048 * 2.0 ** -23 + (64 + 8) * 2.0 ** -24


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def _equal(name, got, ref):
    ref = ref.to(got.dtype)
    assert torch.equal(got, ref), f"{name}: {(got != ref).sum().item()} of {got.numel()} differ"


# tokens, hidden or feed-forward width so long that the weights' gradients, grad_x, y, da or gate and up take
# pieces, on pairs of blocks and on single ones, with rows off 16 bytes and with two-number operands
@pytest.mark.parametrize("T,D,F", [(300000, 24, 40), (300001, 21, 43), (40000, 1100, 1056), (2100, 1032, 16904), (1500, 1500, 33000),
                                   (1100, 70000, 1104), (300, 40, 140000), (40, 264, 270000), (40, 21, 270001), (1, 24, 270000)])
@pytest.mark.parametrize("type_", ["bf16", "fp16"])
def test_whole_numbers(T, D, F, type_):
    """Gates of 32 and more, where act(g) = g and act'(g) = 1 in FP32; every product is a whole number
    below 2^24, exact in FP32 in any order."""
    dtype = M.TYPES[type_]
    g = torch.Generator(device=DEV).manual_seed(T + D + F)

    def few(*s, p=2 / 3):
        u = torch.rand(*s, generator=g, device=DEV)
        return ((u < p / 2).to(dtype) - (u > 1 - p / 2).to(dtype))

    x, dy, wd = few(T, D), few(T, D, p=min(2 / 3, 24 / D)), few(D, F)
    wg, wu = few(F, D, p=min(2 / 3, 24 / D)), few(F, D, p=min(2 / 3, 24 / D))
    x[:, 0], wg[:, 0] = 1.0, 64.0
    y, dx = torch.empty_like(x), torch.empty_like(x)
    gate, up = (torch.empty(T, F, dtype=dtype, device=DEV) for _ in range(2))
    grads = [torch.empty(w.shape, device=DEV) for w in (wg, wu, wd)]
    ws = torch.empty(max(m.mhc_ffn_forward_workspace_bytes(T, D, F), m.mhc_ffn_backward_workspace_bytes(T, D, F)),
                     dtype=torch.uint8, device=DEV)
    m.mhc_ffn_forward(x, wg, wu, wd, y, ws, gate, up)
    d = lambda t: t.double()  # noqa: E731
    rg, ru = d(x) @ d(wg).t(), d(x) @ d(wu).t()
    assert rg.min() >= 32 and rg.max() <= 96 and ru.abs().max() <= 48, "the recipe's ranges"
    _equal("gate", gate, rg)
    _equal("up", up, ru)
    a = rg * ru
    y_ref = (a if T <= 64 else d(a.to(dtype))) @ d(wd).t()
    assert y_ref.abs().max() < 2 ** 24
    _equal("y", y, y_ref.float())
    # the backward on gates of 64 and ups of -1, 0, 1: dg, du and a are exact in eight bits
    gate.fill_(64.0)
    up.copy_(few(T, F))
    m.mhc_ffn_backward(x, wg, wu, wd, gate, up, dy, dx, *grads, ws)
    da = d(dy) @ d(wd)
    assert da.abs().max() <= 64
    dg, du = da * d(up), da * 64
    wg_, wu_ = d(wg), d(wu)
    ref = dg @ wg_ + du @ wu_
    assert ref.abs().max() < 2 ** 24
    _equal("grad_x", dx, ref.float())
    for name, got, r in zip(("grad_w_gate", "grad_w_up", "grad_w_down"), grads, (dg.t() @ d(x), du.t() @ d(x), d(dy).t() @ (64 * d(up)))):
        assert r.abs().max() < 2 ** 24
        _equal(name, got, r)


@pytest.mark.parametrize("T,D,F", [(1 << 23, 16, 16), ((1 << 24) - 5, 8, 13)])
def test_gradients_of_many_tokens(T, D, F):
    """Gradients whose terms are all positive, over up to the most tokens that a call takes.  (Their roundings to
    BF16, 2^-8 at most and as often up as down, come to 2^-8 / sqrt(T) of the sum; 2^-16 leaves room for
    what the activation and its derivative are off.)"""
    g = torch.Generator(device=DEV).manual_seed(T + F)
    positive = lambda *s: (0.5 + torch.rand(*s, generator=g, device=DEV)).to(BF)  # noqa: E731
    x, dy, gate, up = positive(T, D), positive(T, D), positive(T, F), positive(T, F)
    wg, wu, wd = positive(F, D), positive(F, D), positive(D, F)
    grads = [torch.empty(w.shape, device=DEV) for w in (wg, wu, wd)]
    ws = torch.empty(m.mhc_ffn_backward_workspace_bytes(T, D, F), dtype=torch.uint8, device=DEV)
    m.mhc_ffn_backward(x, wg, wu, wd, gate, up, dy, None, *grads, ws)
    ref = [torch.zeros(w.shape, dtype=torch.float64, device=DEV) for w in (wg, wu, wd)]
    for i in range(0, T, 1 << 20):
        xs, ds, gs, us = (t[i:i + (1 << 20)].double() for t in (x, dy, gate, up))
        q = torch.sigmoid(gs)
        da = ds @ wd.double()
        ref[0] += (da * us * q * (1 + gs * (1 - q))).t() @ xs
        ref[1] += (da * gs * q).t() @ xs
        ref[2] += ds.t() @ (gs * q * us)
    for name, got, r in zip(("grad_w_gate", "grad_w_up", "grad_w_down"), grads, ref):
        off = ((got.double() - r) / r).abs().max().item()
        assert off <= SUM + 2.0 ** -16, f"{name}: {off}"


@pytest.mark.parametrize("T,F", [(1024, 1024), (300, 24)])
def test_projections_of_long_rows(T, F):
    """gate and up of 2^20 positive terms each, in FP16, whose rounding is 2^-11 of the value at most."""
    D = 1 << 20
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.rand(T, D, generator=g, device=DEV, dtype=FP) + 0.5
    wg, wu = ((torch.rand(F, D, generator=g, device=DEV, dtype=FP) + 0.5) * 2.0 ** -8 for _ in range(2))
    wd = torch.zeros(D, F, dtype=FP, device=DEV)
    y = torch.empty_like(x)
    gate, up = (torch.empty(T, F, dtype=FP, device=DEV) for _ in range(2))
    ws = torch.empty(m.mhc_ffn_forward_workspace_bytes(T, D, F), dtype=torch.uint8, device=DEV)
    m.mhc_ffn_forward(x, wg, wu, wd, y, ws, gate, up)
    rows = torch.tensor([0, 1, T // 2, T - 1], device=DEV)
    for name, got, w in (("gate", gate, wg), ("up", up, wu)):
        ref = sum(x[rows, i:i + (1 << 16)].double() @ w[:, i:i + (1 << 16)].double().t() for i in range(0, D, 1 << 16))
        off = ((got[rows].double() - ref) / ref).abs().max().item()
        assert off <= 2.0 ** -11 + SUM, f"{name}: {off}"
        # the roundings go up as often as down: what stays on average is the sums'
        assert ((got[rows].double() - ref) / ref).mean().abs().item() <= SUM + 2.0 ** -11 / (4 * F) ** 0.5


@pytest.mark.parametrize("tall", [False, True])
def test_orthogonalised_update_of_long_rows(tall):
    """A short side of 40: A's diagonal is a sum of 2^20 squares."""
    shape = ((1 << 20), 40) if tall else (40, 1 << 20)
    G = torch.randn(*shape, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV)
    G += 3 * torch.randn(shape[0], 1, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)) * (
        torch.randn(1, shape[1], device=DEV, generator=torch.Generator(device=DEV).manual_seed(3)))
    out = torch.empty(*shape, dtype=BF, device=DEV)
    ws = torch.empty(m.mhc_orthogonalize_workspace_bytes(*shape), dtype=torch.uint8, device=DEV)
    m.mhc_orthogonalize(G, out, ws)
    X = G.double() / (G.double().norm() + 1e-7)
    X = X.t() if tall else X
    for _ in range(5):
        A = X @ X.t()
        X = 3.4445 * X + (-4.7750 * A + 2.0315 * (A @ A)) @ X
    M.orthogonal_within(f"{shape}", out, f64(X.t() if tall else X))
