"""Inputs and checks shared by the operators' GPU tests and the checked-build
child (not a test module).  Inputs are drawn on the CPU from a seed; every
check compares with oracle/mhcs_oracle.py within the bound derived there.

Chains (the most additions any term of a result passes through): a row of D
elements is summed by at least 32 threads, so a thread adds at most D / 32 of
them and the threads' sums are joined in at most 10 more steps; with the few
operations that form a term and the final ones, 64 + D / 32 covers every row
statistic and dot product.  Parameter gradients add T rows: 64 + T."""
import numpy as np
import torch

import oracle.mhcs_oracle as S
import rms_backward_gb300 as m

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
RNG = (0x0123456789ABCDEF, 2**63 - 3)   # the step's sum with a sequence number passes 2^63


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def gates(g, T):
    l = torch.randn(T, 24, generator=g)
    r = torch.softmax(l[:, 8:].reshape(T, 4, 4), 2)
    return torch.cat([torch.sigmoid(l[:, :4]), 2 * torch.sigmoid(l[:, 4:8]), r.reshape(T, 16)], 1).contiguous()


def rng_state():
    return torch.tensor([RNG[0], RNG[1]], dtype=torch.int64, device=DEV)


def empty(*shape, dtype=torch.float32):
    """An output full of NaN, so that what is not written shows."""
    return torch.full(shape, float("nan"), dtype=dtype, device=DEV)


def scratch(nbytes):
    return torch.full((max(nbytes, 1),), 0xFF, dtype=torch.uint8, device=DEV)[:nbytes]   # NaN as FP32


def np64(t):
    return t.detach().double().cpu().numpy()


def row_chain(D):
    return 64 + -(-D // 32)


def check(name, got, ref, mag, chain, out="fp32"):
    ok, worst = S.within(np64(got), ref, mag, chain, out)
    assert ok, f"{name}: {worst:.3g} times the bound"


def off_by(t, offset):
    """A contiguous copy on the GPU that starts `offset` elements past an allocation's start."""
    flat = torch.empty(t.numel() + offset, dtype=t.dtype, device=DEV)[offset:]
    return flat.view(t.shape).copy_(t)


# ---------------------------------------------------------------- embedding
def embed_forward_case(T, V, D, n, type_, wide, seed, scale=0.7, offset=0):
    g = gen(seed)
    table = normal(g, V, D, dtype=DTYPES[type_])
    ids = torch.randint(-1, V + 1, (T,), generator=g, dtype=torch.int64 if wide else torch.int32)
    x = off_by(empty(T, n * D, dtype=torch.bfloat16), 3 * offset)
    m.mhc_embed_forward(off_by(ids, offset), off_by(table, offset), x, scale=scale)
    ref = S.embed_forward(ids.numpy(), np64(table), n, scale)
    check("x", x, ref, np.abs(ref), 2, "bf16")


def embed_backward_case(T, V, D, n, wide, accumulate, seed, skew=False, scale=0.7, offset=0):
    g = gen(seed)
    ids = torch.randint(-1, V + 1, (T,), generator=g, dtype=torch.int64 if wide else torch.int32)
    if skew:   # most tokens are one id, some its neighbours
        ids[torch.rand(T, generator=g) < 0.8] = V // 2
    gx = normal(g, T, n * D, dtype=torch.bfloat16)
    start = normal(g, V, D) if accumulate else None
    out = off_by(start if accumulate else empty(V, D), offset)
    ws = scratch(m.mhc_embed_workspace_bytes(T, V, D))
    m.mhc_embed_backward(off_by(ids, offset), off_by(gx, 3 * offset), out, ws, scale=scale, accumulate=accumulate)
    ref, mag, chain = S.embed_backward(ids.numpy(), np64(gx), V, D, scale, None if start is None else np64(start))
    check("grad_table", out, ref, mag, chain)
    if not accumulate:
        none = np.setdiff1d(np.arange(V), ids.numpy())
        assert not out[torch.from_numpy(none).to(DEV)].any()


# ---------------------------------------------------------------- norms
def strided(t, pad):
    """The same values with `pad` more elements between rows (0: compact)."""
    if pad == 0:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def norm_forward_case(T, D, type_, seed, affine=True, stats=True, pad=0, eps=1e-5):
    g = gen(seed)
    x = normal(g, T, D, dtype=DTYPES[type_]) + (torch.randn(T, 1, generator=g) * 3).to(DTYPES[type_])
    gamma, beta = (normal(g, D), normal(g, D)) if affine else (None, None)
    xd, y = strided(x.to(DEV), pad), strided(empty(T, D, dtype=DTYPES[type_]), 2 * pad)
    mean, rstd = (empty(T), empty(T)) if stats else (None, None)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    m.mhc_layernorm_forward(xd, dev(gamma), dev(beta), y, mean, rstd, eps=eps)
    ref = S.norm_forward(np64(x), np64(gamma) if affine else np.ones(D), np64(beta) if affine else np.zeros(D), eps)
    check("y", y, ref[0], ref[3], 2 * row_chain(D), type_)
    if stats:
        check("mean", mean, ref[1], ref[4], row_chain(D))
        check("rstd", rstd, ref[2], ref[5], row_chain(D))


def norm_backward_case(T, D, type_, seed, affine=True, params="both", pad=0, accumulate=False):
    g = gen(seed)
    dt = DTYPES[type_]
    x, gy = normal(g, T, D, dtype=dt), normal(g, T, D, dtype=dt)
    gamma = normal(g, D) if affine else None
    _, mean, rstd, *_ = S.norm_forward(np64(x), 1.0, 0.0, 1e-5)
    mean, rstd = (torch.from_numpy(a).float() for a in (mean, rstd))
    gx = strided(empty(T, D, dtype=dt), 3 * pad)
    start = [normal(g, D), normal(g, D)]
    grads = [None if params == "none" or (params == "beta" and i == 0)
             else s.to(DEV) if accumulate else empty(D) for i, s in enumerate(start)]
    ws = scratch(m.mhc_layernorm_workspace_bytes(T, D)) if params != "none" else None
    m.mhc_layernorm_backward(strided(x.to(DEV), pad), strided(gy.to(DEV), 2 * pad),
                             None if gamma is None else gamma.to(DEV), mean.to(DEV), rstd.to(DEV), gx, grads[0],
                             grads[1], ws, accumulate=accumulate)
    ref, mag = S.norm_backward(np64(x), np64(gy), 1.0 if gamma is None else np64(gamma), np64(mean), np64(rstd))
    check("grad_x", gx, ref[0], mag[0], 2 * row_chain(D), type_)
    for i, name in enumerate(("grad_gamma", "grad_beta")):
        if grads[i] is not None:
            add = np64(start[i]) if accumulate else 0.0
            check(name, grads[i], ref[1 + i] + add, mag[1 + i] + np.abs(add), 64 + T)


def collapse_case(T, D, seed, residual=True, params=True, affine=True, accumulate=False):
    """Forward, and backward from the oracle's statistics."""
    g = gen(seed)
    bf = torch.bfloat16
    x, gy, go = normal(g, T, 4 * D, dtype=bf), normal(g, T, D, dtype=bf), normal(g, T, 4 * D, dtype=bf)
    h = gates(g, T)
    gamma, beta = (normal(g, D), normal(g, D)) if affine else (None, None)
    dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    xd, hd = x.to(DEV), h.to(DEV)
    y, mean, rstd = empty(T, D, dtype=bf), empty(T), empty(T)
    m.mhc_collapse_norm_forward(xd, hd, dev(gamma), dev(beta), y, mean, rstd)
    u, umag = S.collapse(np64(x), np64(h))
    gam = np64(gamma) if affine else np.ones(D)
    ref = S.norm_forward(u, gam, np64(beta) if affine else np.zeros(D), 1e-5, umag)
    check("y", y, ref[0], ref[3], 2 * row_chain(D), "bf16")
    check("mean", mean, ref[1], ref[4], row_chain(D))
    check("rstd", rstd, ref[2], ref[5], row_chain(D))
    mean, rstd = (torch.from_numpy(a).float() for a in (ref[1], ref[2]))
    gx, gh = empty(T, 4 * D, dtype=bf), torch.full((T, 24), 7.0, device=DEV)
    start = [normal(g, D), normal(g, D)]
    gg, gb = (s.to(DEV) if accumulate else empty(D) for s in start) if params else (None, None)
    ws = scratch(m.mhc_collapse_norm_workspace_bytes(T, D)) if params else None
    m.mhc_collapse_norm_backward(xd, hd, gy.to(DEV), dev(gamma), mean.to(DEV), rstd.to(DEV), gx, gh, gg, gb, ws,
                                 grad_x_out=go.to(DEV) if residual else None, accumulate=accumulate)
    ref, mag = S.collapse_norm_backward(np64(x), np64(h), np64(gy), gam, np64(mean), np64(rstd),
                                        np64(go) if residual else None)
    check("grad_x", gx, ref[0], mag[0], 2 * row_chain(D), "bf16")
    check("grad_h", gh[:, :4], ref[1], mag[1], 2 * row_chain(D))
    assert bool((gh[:, 4:] == 7.0).all())
    if params:
        add = [np64(s) if accumulate else 0.0 for s in start]
        check("grad_gamma", gg, ref[2] + add[0], mag[2] + np.abs(add[0]), 64 + T)
        check("grad_beta", gb, ref[3] + add[1], mag[3] + np.abs(add[1]), 64 + T)


# ---------------------------------------------------------------- dropout and update
def dropout_case(shape, type_, p, seed, in_place=False, sequence=9, offset=0):
    g = gen(seed)
    x = normal(g, *shape, dtype=DTYPES[type_])
    n = x.numel()
    xd = torch.zeros(n + offset, dtype=x.dtype, device=DEV)[offset:].view(shape)   # offset elements off the alignment
    xd.copy_(x)
    y = xd if in_place else torch.full((n + offset,), float("nan"), dtype=x.dtype, device=DEV)[offset:].view(shape)
    m.mhc_dropout(xd, y, rng_state(), p=p, sequence=sequence)
    keep = torch.from_numpy(S.keep_mask(shape, p, RNG, sequence))
    want = torch.where(keep, (x.float() * np.float32(S.keep_scale(p))).to(x.dtype), torch.zeros((), dtype=x.dtype))
    assert torch.equal(y.cpu(), want)   # the same FP32 product and rounding: the same bits


def update_case(T, D, p, seed, in_place=False, sequence=4):
    g = gen(seed)
    bf = torch.bfloat16
    x, y, go = normal(g, T, 4 * D, dtype=bf), normal(g, T, D, dtype=bf), normal(g, T, 4 * D, dtype=bf)
    h = gates(g, T)
    xd, yd, hd, state = x.to(DEV), y.to(DEV), h.to(DEV), rng_state() if p else None
    gy, gh = empty(T, D, dtype=bf), torch.full((T, 24), 7.0, device=DEV)
    m.mhc_update_backward(xd, yd, hd, go.to(DEV), gy, gh, state, p=p, sequence=sequence)
    out = xd if in_place else empty(T, 4 * D, dtype=bf)
    m.mhc_update_forward(xd, yd, hd, out, state, p=p, sequence=sequence)
    ref, mag = S.update_forward(np64(x), np64(y), np64(h), p, RNG, sequence)
    check("x_out", out, ref, mag, 16, "bf16")
    (rgy, rgh), (mgy, mgh) = S.update_backward(np64(x), np64(y), np64(h), np64(go), p, RNG, sequence)
    check("grad_y", gy, rgy, mgy, 16, "bf16")
    check("grad_h", gh[:, 4:], rgh, mgh, row_chain(D))
    assert bool((gh[:, :4] == 7.0).all())
