"""CPU oracle of the operators around the projection stage -- TEST INFRASTRUCTURE ONLY.

Embedding into the residual streams, layer norm, counter-based dropout, stream
collapse with its norm, stream update, and their gradients, in FP64 numpy
straight from the definitions in include/mhcpb.h.  The library never imports
this; nothing here is shared with the CUDA path.

Beside each value stands the magnitude its FP32 evaluation is bounded by (the
sum of the absolute values of the terms it adds up, products included).  A
sum of k terms in FP32, in any order in which no term passes through more than
c additions, is off by at most about c 2^-24 times the sum of the terms'
magnitudes; `within` holds results to that plus the rounding of the output
type (2^-8 of the value for BF16, 2^-11 for FP16, 2^-24 for FP32).
"""
from __future__ import annotations

import numpy as np

N = 4
U32 = 2.0 ** -24
ROUND = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "fp16": 2.0 ** -24, "fp32": 2.0 ** -149}   # smallest subnormal


def within(got, ref, mag, chain, out="fp32"):
    """(all within the bound, worst error / bound)."""
    got, ref, mag = (np.asarray(a, dtype=np.float64) for a in (got, ref, mag))
    if got.shape != ref.shape:
        return False, np.inf
    if got.size == 0:
        return True, 0.0
    err32 = chain * U32 * np.broadcast_to(mag, ref.shape)
    lim = err32 + ROUND[out] * (np.abs(ref) + err32) + TINY[out]
    err = np.abs(got - ref)
    ok = np.isfinite(got) & (err <= lim)
    return bool(ok.all()), float(np.max(np.where(np.isfinite(got), err / lim, np.inf)))


# ------------------------------------------------------------------ generator
def philox(counter, key):
    """Philox4x32-10 of one 128-bit counter (four 32-bit words) and a 64-bit key
    (two words), in Python integers (Salmon et al., SC 2011)."""
    c, k = [int(v) for v in counter], [int(v) for v in key]
    for _ in range(10):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF, (p0 >> 32) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def random_words(count, rng, sequence=0):
    """The first `count` words of the stream of rng = (key, step) and a sequence number."""
    key, step = int(rng[0]) % 2**64, (int(rng[1]) + int(sequence)) % 2**64
    out = np.empty((count + 3) // 4 * 4, dtype=np.uint64)
    for i in range(len(out) // 4):
        out[4 * i:4 * i + 4] = philox((i & 0xFFFFFFFF, i >> 32, step & 0xFFFFFFFF, step >> 32),
                                      (key & 0xFFFFFFFF, key >> 32))
    return out[:count]


def keep_mask(shape, p, rng, sequence=0):
    if p == 0:
        return np.ones(shape, dtype=bool)
    threshold = int(np.floor(float(np.float32(p)) * 2.0**32 + 0.5))
    return (random_words(int(np.prod(shape)), rng, sequence) >= threshold).reshape(shape)


def keep_scale(p):
    """1 / (1 - p) as the FP32 value the operators multiply by."""
    return float(np.float32(1.0) / (np.float32(1.0) - np.float32(p)))


def dropout(x, p, rng, sequence=0):
    return np.where(keep_mask(x.shape, p, rng, sequence), np.asarray(x, dtype=np.float64) * keep_scale(p), 0.0)


# ------------------------------------------------------------------ embedding
def embed_forward(ids, table, n_streams, scale):
    t = np.asarray(table, dtype=np.float64)
    ok = (ids >= 0) & (ids < t.shape[0])
    rows = np.where(ok[:, None], t[np.where(ok, ids, 0)] * float(np.float32(scale)), 0.0)
    return np.concatenate([rows] * n_streams, axis=1)


def embed_backward(ids, grad_x, V, D, scale, start=None):
    """(gradient, magnitude, chain per row): the longest chain of additions of a row."""
    g = np.asarray(grad_x, dtype=np.float64).reshape(len(ids), np.shape(grad_x)[1] // D, D)
    out = np.zeros((V, D)) if start is None else np.asarray(start, dtype=np.float64).copy()
    mag, count = np.abs(out), np.zeros((V, 1))
    s = float(np.float32(scale))
    for t, v in enumerate(ids):
        if 0 <= v < V:
            out[v] += s * g[t].sum(0)
            mag[v] += abs(s) * np.abs(g[t]).sum(0)
            count[v] += g.shape[1]
    return out, mag, count + 4


# ------------------------------------------------------------------ norms
def _gate_parts(h):
    h = np.asarray(h, dtype=np.float64)
    return h[:, :4], h[:, 4:8], h[:, 8:].reshape(-1, 4, 4)


def _split(x):
    x = np.asarray(x, dtype=np.float64)
    return x.reshape(x.shape[0], N, -1)


def collapse(x, h):
    """u and the magnitude of its four terms."""
    pre, terms = _gate_parts(h)[0], _split(x)
    return (pre[:, :, None] * terms).sum(1), np.abs(pre[:, :, None] * terms).sum(1)


def norm_forward(u, gamma, beta, eps, umag=None):
    """y, mean, rstd, and the magnitudes of y, of mean and (relative) of rstd."""
    u = np.asarray(u, dtype=np.float64)
    umag = np.abs(u) if umag is None else umag
    mean = u.mean(1)
    var = ((u - mean[:, None]) ** 2).mean(1)
    rstd = 1.0 / np.sqrt(var + eps)
    z = (u - mean[:, None]) * rstd[:, None]
    row = umag.mean(1)
    zmag = (umag + row[:, None]) * rstd[:, None]
    # an error of e in every u moves rstd by at most rstd^2 * e * mean |z| <= rstd * (rstd e)
    rel = 1.0 + rstd * row
    y = z * gamma + beta
    return y, mean, rstd, (zmag + np.abs(z) * rel[:, None]) * np.abs(gamma) + np.abs(beta), row, rstd * rel


def norm_backward(u, gy, gamma, mean, rstd, umag=None):
    """du, dgamma, dbeta from the given mean and rstd, and their magnitudes."""
    u, gy = np.asarray(u, dtype=np.float64), np.asarray(gy, dtype=np.float64)
    mean, rstd = (np.asarray(a, dtype=np.float64)[:, None] for a in (mean, rstd))
    umag = np.abs(u) if umag is None else umag
    z, zmag = (u - mean) * rstd, (umag + np.abs(mean)) * rstd
    w = gy * gamma
    du = rstd * (w - w.mean(1, keepdims=True) - z * (w * z).mean(1, keepdims=True))
    aw = np.abs(w)
    dumag = rstd * (aw + aw.mean(1, keepdims=True) + zmag * (aw * zmag).mean(1, keepdims=True))
    return (du, (gy * z).sum(0), gy.sum(0)), (dumag, (np.abs(gy) * zmag).sum(0), np.abs(gy).sum(0))


def collapse_norm_backward(x, h, gy, gamma, mean, rstd, grad_x_out=None):
    """(grad_x, grad_h[:, :4], dgamma, dbeta) and their magnitudes."""
    pre, _, res = _gate_parts(h)
    xs = _split(x)
    u, umag = collapse(x, h)
    (du, gg, gb), (dumag, ggm, gbm) = norm_backward(u, gy, gamma, mean, rstd, umag)
    gx = pre[:, :, None] * du[:, None, :]
    gxm = np.abs(pre)[:, :, None] * dumag[:, None, :]
    if grad_x_out is not None:
        go = _split(grad_x_out)
        gx = gx + np.einsum("tij,tid->tjd", res, go)
        gxm = gxm + np.einsum("tij,tid->tjd", np.abs(res), np.abs(go))
    gh = (xs * du[:, None, :]).sum(2)
    ghm = (np.abs(xs) * dumag[:, None, :]).sum(2)
    T = gx.shape[0]
    return (gx.reshape(T, -1), gh, gg, gb), (gxm.reshape(T, -1), ghm, ggm, gbm)


# ------------------------------------------------------------------ stream update
def update_forward(x, y, h, p=0.0, rng=None, sequence=0):
    _, post, res = _gate_parts(h)
    xs, yd = _split(x), dropout(y, p, rng, sequence)
    out = np.einsum("tij,tjd->tid", res, xs) + post[:, :, None] * yd[:, None, :]
    mag = np.einsum("tij,tjd->tid", np.abs(res), np.abs(xs)) + np.abs(post)[:, :, None] * np.abs(yd)[:, None, :]
    return out.reshape(out.shape[0], -1), mag.reshape(out.shape[0], -1)


def update_backward(x, y, h, grad_x_out, p=0.0, rng=None, sequence=0):
    """(grad_y, grad_h[:, 4:]) and their magnitudes."""
    _, post, _ = _gate_parts(h)
    xs, go, yd = _split(x), _split(grad_x_out), dropout(y, p, rng, sequence)
    f = np.where(keep_mask(yd.shape, p, rng, sequence), keep_scale(p), 0.0)
    gy = f * (post[:, :, None] * go).sum(1)
    gym = f * np.abs(post[:, :, None] * go).sum(1)
    T = gy.shape[0]
    gh = np.concatenate([(go * yd[:, None, :]).sum(2), np.einsum("tid,tjd->tij", go, xs).reshape(T, 16)], 1)
    ghm = np.concatenate([np.abs(go * yd[:, None, :]).sum(2),
                          np.einsum("tid,tjd->tij", np.abs(go), np.abs(xs)).reshape(T, 16)], 1)
    return (gy, gh), (gym, ghm)
