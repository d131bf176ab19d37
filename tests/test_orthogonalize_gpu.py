"""The orthogonalised update on the GPU against the formula in FP64."""
import numpy as np
import pytest
import torch

import oracle.mhcm_oracle as O
import rms_backward_gb300 as m

import matrix_cases as M
from matrix_cases import DEV, f64

pytestmark = pytest.mark.gpu
BF = torch.bfloat16

SHAPES = [(1, 20), (8, 4000), (20480, 24), (32, 25000), (32, 30000), (33, 2000), (17, 5), (1, 1), (1, 9), (9, 1), (2, 3), (16, 16), (24, 2048), (2048, 24), (64, 200), (100, 100), (127, 129), (129, 128),
          (257, 130), (300, 1000), (1001, 303), (640, 640)]


@pytest.mark.parametrize("mm,n", SHAPES)
@pytest.mark.parametrize("type_", ["fp32", "bf16", "fp16"])
def test_shapes(mm, n, type_):
    M.orthogonalize_case(mm, n, type_, seed=mm + n)


@pytest.mark.parametrize("mm,n", [(24, 2048), (130, 130), (200, 700), (700, 200), (100, 99)])
@pytest.mark.parametrize("kind", ["strong", "low"])
def test_spectra(mm, n, kind):
    """Few strong directions, and ranks far below the sides: rounding must not
    fill the directions that the matrix leaves empty."""
    M.orthogonalize_case(mm, n, "fp32", kind, seed=mm + n)


@pytest.mark.parametrize("mm,n", [(2300, 2310), (2305, 2600), (2600, 2304)])
def test_large(mm, n):
    M.orthogonalize_case(mm, n, "fp32", "strong", seed=1)


@pytest.mark.parametrize("steps", [1, 2, 3, 4])
def test_steps(steps):
    M.orthogonalize_case(60, 90, "fp32", seed=steps, steps=steps)


@pytest.mark.parametrize("steps", [8, 32])
def test_many_steps(steps):
    """The polynomial moves singular values about within [0.68, 1.21] for ever, and far apart from
    what a slightly different start gives; they stay there, and the directions are G's: out G^T is
    symmetric."""
    G = torch.from_numpy(M.spectrum(60, 90, "gauss", steps)).float().to(DEV)
    ws, _ = M.scratch(m.mhc_orthogonalize_workspace_bytes(60, 90))
    out = torch.empty(60, 90, dtype=BF, device=DEV)
    m.mhc_orthogonalize(G, out, ws, steps=steps)
    s = np.linalg.svd(f64(out), compute_uv=False)
    # the values before the rounding to BF16, which moves each by at most 2^-8 |out|_F < 2^-8 * 1.21 * sqrt(60)
    assert s.min() > 0.68 - 0.037 and s.max() < 1.21 + 0.037
    p = f64(out) @ f64(G).T
    # each step may turn directions by its FP16 operands' error, below 2^-9, and the output's rounding by 2^-8
    assert np.linalg.norm(p - p.T) < 2 * (2.0 ** -8 + steps * 2.0 ** -9) * np.linalg.norm(p)


@pytest.mark.parametrize("mm,n", [(40, 72), (72, 40), (400, 520)])
def test_row_strides_and_scale(mm, n):
    M.orthogonalize_case(mm, n, "fp32", seed=2, pad=8, scale=0.25)
    M.orthogonalize_case(mm, n, "bf16", seed=2, pad=64, scale=-3.0)


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e18, 1e30])
def test_sizes_whose_squares_leave_fp32(size):
    """The result does not depend on G's size while |G| is far above eps."""
    G = torch.from_numpy(M.spectrum(50, 80, "gauss", 1)).float().to(DEV)
    ws, _ = M.scratch(m.mhc_orthogonalize_workspace_bytes(50, 80))
    out = torch.empty(50, 80, dtype=BF, device=DEV)
    m.mhc_orthogonalize(G * size, out, ws, eps=0.0)
    M.orthogonal_within(f"times {size}", out, O.orthogonalize(f64(G), eps=0.0))


def test_one_element_of_another_size():
    """One element far above the others takes the whole norm; the others vanish beside it."""
    G = torch.full((20, 30), 1e-25, device=DEV)
    G[3, 4] = 1e25
    ws, _ = M.scratch(m.mhc_orthogonalize_workspace_bytes(20, 30))
    out = torch.empty(20, 30, dtype=BF, device=DEV)
    m.mhc_orthogonalize(G, out, ws)
    s = 1.0
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    ref = torch.zeros(20, 30)
    ref[3, 4] = s
    assert (out.float().cpu() - ref).abs().max() <= (2.0 ** -8 + 2.0 ** -9) * s


def test_zero_eps_and_non_finite():
    ws, _ = M.scratch(m.mhc_orthogonalize_workspace_bytes(40, 50))
    out = torch.empty(40, 50, dtype=BF, device=DEV)
    G = torch.zeros(40, 50, device=DEV)
    m.mhc_orthogonalize(G, out, ws)
    assert (out == 0).all()
    m.mhc_orthogonalize(G, out, ws, eps=0.0)
    assert torch.isnan(out).all()
    for bad in (float("nan"), float("inf")):
        G = torch.from_numpy(M.spectrum(40, 50, "gauss", 1)).float().to(DEV)
        G[7, 9] = bad
        m.mhc_orthogonalize(G, out, ws)
        assert torch.isnan(out).all()


def test_eps_counts():
    """|G| = 1 with eps = 1: X starts at G / 2."""
    G = torch.from_numpy(M.spectrum(30, 40, "gauss", 1)).float().to(DEV)
    G /= G.norm()
    ws, _ = M.scratch(m.mhc_orthogonalize_workspace_bytes(30, 40))
    out = torch.empty(30, 40, dtype=BF, device=DEV)
    m.mhc_orthogonalize(G, out, ws, eps=1.0)
    M.orthogonal_within("eps", out, O.orthogonalize(f64(G), eps=1.0))


@pytest.mark.parametrize("mm,n", [(24, 2048), (300, 500), (2300, 2310)])
def test_same_bits_again(mm, n):
    G = torch.from_numpy(M.spectrum(mm, n, "strong", 1)).float().to(DEV)
    outs = []
    for fill in (0x00, 0x7F):
        ws = torch.full((m.mhc_orthogonalize_workspace_bytes(mm, n),), fill, dtype=torch.uint8, device=DEV)
        out = torch.empty(mm, n, dtype=BF, device=DEV)
        m.mhc_orthogonalize(G, out, ws)
        outs.append(out)
    assert torch.equal(*outs)
