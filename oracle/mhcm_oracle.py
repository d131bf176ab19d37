"""FP64 reference of the gated feed-forward block, its gradient, and the
orthogonalised update of a matrix, from the formulas in include/mhcpb.h, with
elementwise bounds of what 16-bit operands and FP32 sums may be off.

Bounds.  A rounding to a type is off by at most half a step, HALF of the value
(FP16's denormals: TINY).  A product's FP32 sum over K terms, added on the
tensor cores in groups of 16 that are aligned to their largest term and cut, is
off by at most (K + 64) 2^-23 of the sum of the terms' magnitudes.  exp, erfc and
the division are off by a few units, more for larger arguments (see _act).
"""
from __future__ import annotations

import numpy as np

HALF = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}
A, B, C = 3.4445, -4.7750, 2.0315


def _sum(K):
    return (K + 64) * 2.0 ** -23


def _erfc(v):
    from math import erfc
    return np.vectorize(erfc, otypes=[np.float64])(v) if v.size else v


def _act(g, kind):
    """act(g), act'(g), and how far off FP32 forms of them may be."""
    if kind == "silu":
        with np.errstate(over="ignore"):
            q = 1.0 / (1.0 + np.exp(-g))
        f, d, e = g * q, q * (1.0 + g * (1.0 - q)), (16 + 4 * abs(g)) * 2.0 ** -23
        return f, d, e * abs(f), e * q * (1.0 + abs(g))
    p = 0.5 * _erfc(-g * 0.5 ** 0.5)
    phi = np.exp(-0.5 * g * g) * (2.0 * np.pi) ** -0.5
    e = (16 + 4 * abs(g) + 4 * g * g) * 2.0 ** -23
    # below 2^-126 results lose bits: an absolute share
    return g * p, p + g * phi, e * abs(g * p) + 2.0 ** -120, e * (p + abs(g) * phi) + 2.0 ** -120


def _rounded(v, e, type_):
    """The error bound of a value with bound e after rounding to type_."""
    return e + HALF[type_] * (abs(v) + e) + TINY[type_]


def ffn_forward(x, wg, wu, wd, act, type_):
    """(y, gate, up) and their bounds, from FP64 arrays."""
    D, F = x.shape[1], wg.shape[0]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = (_sum(D) * (abs(x) @ abs(w).T) for w in (wg, wu))
    f, _, ef, _ = _act(g, act)
    ef = ef + 1.13 * eg                              # |act'| <= 1.13
    a = f * u
    ea = _rounded(a, ef * (abs(u) + eu) + abs(f) * eu + 2.0 ** -23 * abs(a), type_)
    y = a @ wd.T
    ey = ea @ abs(wd).T + _sum(F) * ((abs(a) + ea) @ abs(wd).T)
    return (y, g, u), (_rounded(y, ey, type_), _rounded(g, eg, type_), _rounded(u, eu, type_))


def ffn_backward(x, wg, wu, wd, g, u, dy, act, type_, grad_type, before=None):
    """(grad_x, grad_w_gate, grad_w_up, grad_w_down) and their bounds; `before`:
    what the weights' gradients are added to."""
    T, D = x.shape
    F = wg.shape[0]
    da = dy @ wd
    eda = _sum(D) * (abs(dy) @ abs(wd))
    f, d, ef, ed = _act(g, act)
    a, dg, du = f * u, da * u * d, da * f
    ea = _rounded(a, ef * abs(u) + 2.0 ** -22 * abs(a), type_)
    edg = _rounded(dg, eda * abs(u) * (abs(d) + ed) + abs(da * u) * ed + 2.0 ** -21 * abs(dg), type_)
    edu = _rounded(du, eda * (abs(f) + ef) + abs(da) * ef + 2.0 ** -22 * abs(du), type_)
    dx = dg @ wg + du @ wu
    mdg, mdu = abs(dg) + edg, abs(du) + edu
    edx = edg @ abs(wg) + edu @ abs(wu) + _sum(2 * F) * (mdg @ abs(wg) + mdu @ abs(wu))
    out, bound = [dx], [_rounded(dx, edx, type_)]
    for i, (left, eleft, right, eright) in enumerate(((dg, edg, x, 0), (du, edu, x, 0), (dy, 0, a, ea))):
        w = left.T @ right
        ml, mr = abs(left) + eleft, abs(right) + eright
        e = (ml.T @ mr - abs(left).T @ abs(right)) + _sum(T) * (ml.T @ mr)
        if before is not None:
            w = w + before[i]
            e = e + 2.0 ** -24 * (abs(w) + e)
        out.append(w)
        bound.append(_rounded(w, e, grad_type))
    return out, bound


def orthogonalize(g, steps=5, eps=1e-7):
    """X after `steps` steps, from the formula."""
    X = g / (np.sqrt((g * g).sum()) + eps)
    X = X.T if g.shape[0] > g.shape[1] else X
    for _ in range(steps):
        M = X @ X.T
        X = A * X + (B * M + C * (M @ M)) @ X
    return X.T if g.shape[0] > g.shape[1] else X


def _half(v, scale):
    return (v * scale).astype(np.float16).astype(np.float64) / scale


def orthogonalize_rounded(g, steps=5, eps=1e-7):
    """The same with FP16 operands as the library rounds them: X's copy and A at
    2^15 times their value, B at 2^14 times; X itself is kept in FP32, and what the
    diagonals of A and B lose is put back."""
    X = g / (np.sqrt((g * g).sum()) + eps)
    tall = g.shape[0] > g.shape[1]
    X = X.T if tall else X
    for _ in range(steps):
        h = _half(X, 2.0 ** 15)
        M = h @ h.T
        R = _half(M, 2.0 ** 15)
        l = np.diag(M) - np.diag(R)
        P = C * (R @ R) + (B + C * (l[:, None] + l[None])) * R + np.diag((B + C * l) * l)
        Q = _half(P, 2.0 ** 14)
        X = ((A + np.diag(P) - np.diag(Q))[:, None] * X + Q @ h).astype(np.float32).astype(np.float64)
    return X.T if tall else X
