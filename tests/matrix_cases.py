"""Cases of the gated feed-forward block and the orthogonalised update: inputs,
the library's call, and the comparison with the FP64 oracle (used by the GPU
tests and by the bounds-checked run)."""
from __future__ import annotations

import numpy as np
import torch

import oracle.mhcm_oracle as O
import rms_backward_gb300 as m

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(T, D, dtype, pad=0, fill=float("nan")):
    """A [T, D] view with rows D + pad apart, and the buffer it is in (with
    `fill` everywhere)."""
    buf = torch.full((max(T, 1), D + pad), fill, dtype=dtype, device=DEV)
    return buf[:T, :D], buf


def put(values, dtype, pad=0):
    t, _ = rows(*values.shape, dtype, pad)
    t.copy_(values)
    return t


def scratch(size):
    """A workspace whose every byte is a NaN's, and a guard behind it."""
    buf = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device=DEV)
    return buf[:size], buf[size:]


def within(name, got, ref, bound):
    got = f64(got)
    bad = ~(abs(got - ref) <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(np.isnan(got), np.inf, abs(got - ref) / np.maximum(bound, 1e-300))), got.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside; at {i}: {got[i]} for {ref[i]} +- {bound[i]}")


def inputs(T, D, F, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = put(n(T, D), dtype, pad)
    wg, wu, wd = (put(w, dtype) for w in (n(F, D) * D ** -0.5, n(F, D) * D ** -0.5, n(D, F) * F ** -0.5))
    return g, x, wg, wu, wd


def ffn_forward_case(T, D, F, type_, act="silu", train=True, seed=0, pad=0, **kw):
    dtype = TYPES[type_]
    _, x, wg, wu, wd = inputs(T, D, F, dtype, seed, pad)
    y, ybuf = rows(T, D, dtype, pad)
    gate, up = (rows(T, F, dtype)[0] if train else None for _ in range(2))
    ws, guard = scratch(m.mhc_ffn_forward_workspace_bytes(T, D, F))
    m.mhc_ffn_forward(x, wg, wu, wd, y, ws, gate, up, activation=act, **kw)
    torch.cuda.synchronize()
    ref, bound = O.ffn_forward(*map(f64, (x, wg, wu, wd)), act, type_)
    for name, got, r, b in zip(("y", "gate", "up"), (y, gate, up), ref, bound):
        if got is not None:
            within(f"{name} T={T} D={D} F={F} {type_} {act}", got, r, b)
    assert torch.isnan(ybuf[:, D:]).all() and (guard == 0xFF).all()
    return x, wg, wu, wd, y, gate, up


def ffn_backward_case(T, D, F, type_, act="silu", grad_type=None, accumulate=False, seed=0, pad=0, which=(1, 1, 1, 1), **kw):
    dtype, grad_type = TYPES[type_], grad_type or type_
    g, x, wg, wu, wd = inputs(T, D, F, dtype, seed, pad)
    gate, up = (put(2 * torch.randn(T, F, generator=g), dtype) for _ in range(2))
    dy = put(torch.randn(T, D, generator=g), dtype, pad)
    dx, dxbuf = rows(T, D, dtype, pad)
    shapes = ((F, D), (F, D), (D, F))
    before = [torch.randn(*s, generator=g).to(TYPES[grad_type]).to(DEV) for s in shapes]
    grads = [b.clone() if accumulate else torch.full_like(b, float("nan")) for b in before]
    ws, guard = scratch(m.mhc_ffn_backward_workspace_bytes(T, D, F))
    out = [t if w else None for t, w in zip([dx, *grads], which)]
    m.mhc_ffn_backward(x, wg, wu, wd, gate, up, dy, *out, ws, activation=act, accumulate=accumulate, **kw)
    torch.cuda.synchronize()
    ref, bound = O.ffn_backward(*map(f64, (x, wg, wu, wd, gate, up, dy)), act, type_, grad_type,
                                [f64(b) for b in before] if accumulate else None)
    for name, got, r, b in zip(("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down"), out, ref, bound):
        if got is not None:
            within(f"{name} T={T} D={D} F={F} {type_}/{grad_type} {act}", got, r, b)
    for t, w, b in zip([dx, *grads], which, [None, *before]):   # what was not asked for is left alone
        if not w:
            assert torch.equal(t, b) if b is not None and accumulate else torch.isnan(t).all()
    assert torch.isnan(dxbuf[:, D:]).all() and (guard == 0xFF).all()


def _round(v, type_):
    return torch.from_numpy(v).float().to(TYPES[type_]).double().numpy()


def ffn_exact_case(T, D, F, type_, seed=0, grad_type="fp32"):
    """Whole numbers throughout: every gate is at least 32, where act(g) = g and
    act'(g) = 1 in FP32, so each output is one rounding of a whole number.  Up to
    64 tokens what the rounding of a, dg and du loses is kept (two numbers of 8 bits
    hold the 16 that these have), but for the weights' gradients."""
    dtype = TYPES[type_]
    g = np.random.default_rng(seed)
    few = lambda *s, p: g.choice([-1.0, 0.0, 1.0], s, p=[p / 2, 1 - p, p / 2])  # noqa: E731
    p = min(0.5, 24 / max(D, F))
    x, dy = few(T, D, p=0.5), few(T, D, p=p)
    x[:, 0] = 1.0
    wg, wu, wd = few(F, D, p=p), few(F, D, p=p), few(D, F, p=p)
    wg[:, 0] = 64.0
    gate, up = x @ wg.T, x @ wu.T
    assert gate.min() >= 32 and gate.max() <= 96 and abs(up).max() <= 40, "the recipe's ranges"
    t = lambda v: torch.from_numpy(v).to(dtype).to(DEV)  # noqa: E731
    xt, wgt, wut, wdt, dyt = t(x), t(wg), t(wu), t(wd), t(dy)
    y, gt, ut = (rows(T, n, dtype)[0] for n in (D, F, F))
    ws, _ = scratch(m.mhc_ffn_forward_workspace_bytes(T, D, F))
    m.mhc_ffn_forward(xt, wgt, wut, wdt, y, ws, gt, ut)
    a, few = _round(gate * up, type_), T <= 64
    assert abs(gate * up).max() < 2 ** 16
    for name, got, ref in (("gate", gt, gate), ("up", ut, up), ("y", y, _round((gate * up if few else a) @ wd.T, type_))):
        assert np.array_equal(f64(got), ref), f"{name} T={T} D={D} F={F} {type_}: {(f64(got) != ref).sum()} of {ref.size} differ"
    da = dy @ wd
    dg, du = _round(da * up, type_), _round(da * gate, type_)
    dx = rows(T, D, dtype)[0]
    grads = [rows(*s, TYPES[grad_type])[0] for s in ((F, D), (F, D), (D, F))]
    ws, _ = scratch(m.mhc_ffn_backward_workspace_bytes(T, D, F))
    m.mhc_ffn_backward(xt, wgt, wut, wdt, gt, ut, dyt, dx, *grads, ws)
    assert max(abs(da * up).max(), abs(da * gate).max()) < 2 ** 16
    dx_ref = (da * up) @ wg + (da * gate) @ wu if few else dg @ wg + du @ wu
    ref = [_round(dx_ref, type_), *(_round(v, grad_type) for v in (dg.T @ x, du.T @ x, dy.T @ a))]
    for name, got, r in zip(("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down"), (dx, *grads), ref):
        assert abs(r).max() < 2 ** 24
        assert np.array_equal(f64(got), r), f"{name} T={T} D={D} F={F} {type_}: {(f64(got) != r).sum()} of {r.size} differ"


def spectrum(mm, n, kind, seed):
    """Matrices with all directions alike, few strong ones over noise, or a low rank."""
    g = np.random.default_rng(seed)
    if kind == "gauss":
        return g.standard_normal((mm, n))
    r = max(1, min(mm, n, 64) // 4)
    low = (g.standard_normal((mm, r)) * np.arange(1, r + 1) ** -0.75) @ g.standard_normal((r, n))
    return low if kind == "low" else low + 0.1 * g.standard_normal((mm, n))


def orthogonal_within(name, out, ref):
    """out against the formula's result, after at most five steps.  FP16 operands move it by
    less than 2^-9 of its 2-norm (the oracle with those roundings is held to that).
    Which way single roundings fall depends on the FP32 sums before them, and a
    rounding of one step decides those of the next, so elements are held to the
    errors' spread: a root mean square of at most 2^-9 of the result's, eight times
    that for the farthest of up to ten million elements (a normal error passes 8
    deviations once in 10^15).  The output's own rounding adds 2^-8 of the element."""
    norm = np.linalg.norm(ref)
    off = np.linalg.norm(f64(out) - ref)
    assert off <= (2.0 ** -8 + 2.0 ** -9) * norm, f"{name}: {off / norm}"
    within(name, out, ref, 2.0 ** -8 * abs(ref) + 2.0 ** -6 * norm / np.sqrt(ref.size))


def orthogonalize_case(mm, n, type_, kind="gauss", seed=0, pad=0, steps=5, scale=1.0, size=1.0):
    """Against the formula (see orthogonal_within)."""
    G = put(torch.from_numpy(size * spectrum(mm, n, kind, seed)), TYPES[type_], pad)
    out, buf = rows(mm, n, torch.bfloat16, pad)
    ws, guard = scratch(m.mhc_orthogonalize_workspace_bytes(mm, n))
    m.mhc_orthogonalize(G, out, ws, steps=steps, scale=scale)
    torch.cuda.synchronize()
    orthogonal_within(f"{mm} x {n} {type_} {kind} {steps} steps", out, scale * O.orthogonalize(f64(G), steps))
    assert torch.isnan(buf[:, n:]).all() and (guard == 0xFF).all()
    return G, out
