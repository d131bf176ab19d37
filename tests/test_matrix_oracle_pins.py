"""The FP64 oracle of the feed-forward block and the orthogonalised update, held
to central differences, hand-worked values and what the formulas imply."""
import numpy as np
import pytest

import oracle.mhcm_oracle as O
from matrix_cases import spectrum


def _case(act, T=3, D=4, F=5):
    g = np.random.default_rng(7)
    x, wg, wu, wd, dy = (g.standard_normal(s) for s in ((T, D), (F, D), (F, D), (D, F), (T, D)))
    (y, gate, up), bounds = O.ffn_forward(x, wg, wu, wd, act, "bf16")
    assert all((b > 0).all() for b in bounds)
    return (x, wg, wu, wd), gate, up, dy


def test_by_hand():
    """One token, one column: silu(2) = 2 / (1 + e^-2), gelu(2) = 2 Phi(2)."""
    one = lambda v: np.array([[v]])  # noqa: E731
    (y, g, u), _ = O.ffn_forward(one(1.0), one(2.0), one(3.0), one(0.5), "silu", "bf16")
    assert g == 2 and u == 3 and abs(y - 0.5 * 3 * 1.7615941559557649) < 1e-15
    (y, _, _), _ = O.ffn_forward(one(1.0), one(2.0), one(3.0), one(0.5), "gelu", "bf16")
    assert abs(y - 0.5 * 3 * 1.9544997361036416) < 1e-15


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradient_is_the_differences(act):
    args, gate, up, dy = _case(act)
    grads, bounds = O.ffn_backward(*args, gate, up, dy, act, "bf16", "fp32")
    h = 1e-5
    for k, (a, got) in enumerate(zip(args, grads)):
        for i in np.ndindex(a.shape):
            side = []
            for s in (h, -h):
                b = [v.copy() for v in args]
                b[k][i] += s
                side.append((O.ffn_forward(*b, act, "bf16")[0][0] * dy).sum())
            assert abs((side[0] - side[1]) / (2 * h) - got[i]) < 1e-7
    assert all((b > 0).all() for b in bounds)


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (6, 6)])
def test_singular_values_go_through_the_polynomial(shape):
    g = np.random.default_rng(1).standard_normal(shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / np.linalg.norm(g)
    for _ in range(5):
        s = O.A * s + O.B * s ** 3 + O.C * s ** 5
    assert np.allclose(O.orthogonalize(g, eps=0.0), (u * s) @ vt, atol=1e-12)


def test_bounds_that_keep_fp16_finite():
    """No step takes a singular value in [0, 1] above 1.21, whatever the number of steps, so
    A stays below 1.47 and b t + c t^2 within 2.81 in magnitude."""
    s, top = np.linspace(0, 1, 200001), 1.0
    for _ in range(32):
        s = O.A * s + O.B * s ** 3 + O.C * s ** 5
        assert s.min() >= 0
        top = max(top, s.max())
    wide = np.linspace(0, 1.21, 200001)
    assert top < 1.21 and (O.A * wide + O.B * wide ** 3 + O.C * wide ** 5).max() < 1.21
    t = wide ** 2
    assert t.max() < 1.47 and abs(O.B * t + O.C * t * t).max() < 2.81
    assert 1.21 * 2 ** 15 < 65504 and 1.47 * 2 ** 15 < 65504 and 2 * 2.81 * 2 ** 14 < 2 * 65504


@pytest.mark.parametrize("kind", ["gauss", "strong", "low"])
@pytest.mark.parametrize("shape", [(128, 128), (64, 200), (24, 2000), (300, 40)])
def test_rounding_stays_small(kind, shape):
    """FP16 operands move the result by less than 2^-9 of it, low ranks too."""
    g = spectrum(*shape, kind, 3)
    exact, rounded = O.orthogonalize(g), O.orthogonalize_rounded(g)
    assert np.linalg.norm(rounded - exact) < 2.0 ** -9 * np.linalg.norm(exact)
