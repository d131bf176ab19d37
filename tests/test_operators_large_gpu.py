"""Tensors of more than 2^31 elements, where a 32-bit index would wrap, and
dropout of more than 2^34, whose counters pass 32 bits.  Rows are independent of
one another, so a few of them, before and after the 2^31st element, are compared
with the oracle; parameter gradients are sums over the same rows, the others'
upstream gradient being zero."""
import numpy as np
import pytest
import torch

import oracle.mhcs_oracle as S
import rms_backward_gb300 as m

import operators_cases as C
from operators_cases import DEV, check, empty, gen, normal, np64, rng_state, scratch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LIMIT = 1 << 31


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def _picked(T, width):
    """Rows at both ends and on both sides of elements 2^30, 2^31 and 2^32."""
    rows = {0, 1, T // 3, T - 2, T - 1}
    for e in (1 << 30, LIMIT, 1 << 32):
        rows |= {r for r in (e // width - 1, e // width, e // width + 1) if 0 <= r < T}
    return torch.tensor(sorted(rows))


def _zeros(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


def _with_rows(shape, rows, values):
    t = _zeros(*shape)
    t[rows.to(DEV)] = values.to(DEV)
    return t


def _take(t, rows):
    return t[rows.to(t.device)]


@pytest.mark.parametrize("D", [5120, 5121])   # rows on 16-byte boundaries, and not
def test_norm(D):
    T = LIMIT // D + 500
    g, rows = gen(D), _picked(LIMIT // D + 500, D)
    k = len(rows)
    xr, gyr, gamma, beta = normal(g, k, D, dtype=BF), normal(g, k, D, dtype=BF), normal(g, D), normal(g, D)
    x, gy, y = _with_rows((T, D), rows, xr), _with_rows((T, D), rows, gyr), _zeros(T, D)
    mean, rstd = empty(T), empty(T)
    m.mhc_layernorm_forward(x, gamma.to(DEV), beta.to(DEV), y, mean, rstd)
    ref = S.norm_forward(np64(xr), np64(gamma), np64(beta), 1e-5)
    check("y", _take(y, rows), ref[0], ref[3], 2 * C.row_chain(D), "bf16")
    check("mean", _take(mean, rows), ref[1], ref[4], C.row_chain(D))
    grads = empty(D), empty(D)
    m.mhc_layernorm_backward(x, gy, gamma.to(DEV), mean, rstd, y, *grads, scratch(m.mhc_layernorm_workspace_bytes(T, D)))
    ref, mag = S.norm_backward(np64(xr), np64(gyr), np64(gamma), np64(_take(mean, rows)), np64(_take(rstd, rows)))
    check("grad_x", _take(y, rows), ref[0], mag[0], 2 * C.row_chain(D), "bf16")
    for got, r, a in zip(grads, ref[1:], mag[1:]):
        check("parameters", got, r, a, 64 + T // 152)


@pytest.mark.parametrize("D", [5120, 5121])
def test_streams(D):
    """Collapse and update, each with its gradient, of 2^31 and more stream elements."""
    T = LIMIT // (4 * D) + 500
    g, rows = gen(D), _picked(T, 4 * D)
    k, p, seq = len(rows), 0.3, 4
    xr, gor = normal(g, k, 4 * D, dtype=BF), normal(g, k, 4 * D, dtype=BF)
    yr, gyr, gamma, beta = normal(g, k, D, dtype=BF), normal(g, k, D, dtype=BF), normal(g, D), normal(g, D)
    h = C.gates(g, T)
    x, go, hd, hr = _with_rows((T, 4 * D), rows, xr), _with_rows((T, 4 * D), rows, gor), h.to(DEV), np64(h[rows])
    y, gy = _with_rows((T, D), rows, yr), _with_rows((T, D), rows, gyr)
    out, small, gh = _zeros(T, 4 * D), _zeros(T, D), _zeros(T, 24, dtype=torch.float32)
    mean, rstd, gg, gb = empty(T), empty(T), empty(D), empty(D)

    m.mhc_collapse_norm_forward(x, hd, gamma.to(DEV), beta.to(DEV), small, mean, rstd)
    u, umag = S.collapse(np64(xr), hr)
    ref = S.norm_forward(u, np64(gamma), np64(beta), 1e-5, umag)
    check("y", _take(small, rows), ref[0], ref[3], 2 * C.row_chain(D), "bf16")
    m.mhc_collapse_norm_backward(x, hd, gy, gamma.to(DEV), mean, rstd, out, gh, gg, gb,
                                 scratch(m.mhc_collapse_norm_workspace_bytes(T, D)), grad_x_out=go)
    ref, mag = S.collapse_norm_backward(np64(xr), hr, np64(gyr), np64(gamma), np64(_take(mean, rows)),
                                        np64(_take(rstd, rows)), np64(gor))
    check("grad_x", _take(out, rows), ref[0], mag[0], 2 * C.row_chain(D), "bf16")
    check("grad_h", _take(gh, rows)[:, :4], ref[1], mag[1], 2 * C.row_chain(D))
    check("grad_gamma", gg, ref[2], mag[2], 64 + T // 152)
    check("grad_beta", gb, ref[3], mag[3], 64 + T // 152)

    # the mask of element (t, c) follows from t D + c
    m.mhc_update_forward(x, y, hd, out, rng_state(), p=p, sequence=seq)
    keep = _keep_rows(rows, D, p, seq)
    yd = np.where(keep, np64(yr) * S.keep_scale(p), 0.0)
    ref, mag = S.update_forward(np64(xr), yd, hr)
    check("x_out", _take(out, rows), ref, mag, 16, "bf16")
    m.mhc_update_backward(x, y, hd, go, small, gh, rng_state(), p=p, sequence=seq)
    (rgy, rgh), (mgy, mgh) = S.update_backward(np64(xr), yd, hr, np64(gor))
    f = np.where(keep, S.keep_scale(p), 0.0)
    check("grad_y", _take(small, rows), f * rgy, f * mgy, 16, "bf16")
    check("grad_h", _take(gh, rows)[:, 4:], rgh, mgh, C.row_chain(D))


def _words(first, count, seq):
    """`count` words of the generator from element `first` on."""
    step, key = (C.RNG[1] + seq) % 2**64, C.RNG[0]
    out = []
    for i in range(first // 4, (first + count + 3) // 4):
        out += S.philox((i & 0xFFFFFFFF, i >> 32, step & 0xFFFFFFFF, step >> 32), (key & 0xFFFFFFFF, key >> 32))
    return np.array(out[first % 4:first % 4 + count], dtype=np.uint64)


def _keep_rows(rows, D, p, seq):
    threshold = int(np.floor(float(np.float32(p)) * 2.0**32 + 0.5))
    return np.stack([_words(int(r) * D, D, seq) >= threshold for r in rows])


def _check_dropout(y, value, at, p, seq, count=4099):
    threshold = int(np.floor(float(np.float32(p)) * 2.0**32 + 0.5))
    count = min(count, y.numel() - at)
    want = np.where(_words(at, count, seq) >= threshold, value * S.keep_scale(p), 0.0)
    assert np.array_equal(np64(y[at:at + count]), np64(torch.from_numpy(want).to(y.dtype)))


@pytest.mark.parametrize("n,offset", [(LIMIT + 4097, 0), (LIMIT + 4097, 1), ((1 << 34) + 100003, 0)])
def test_dropout(n, offset):
    """In place; above 2^34 elements the counter's low half passes 32 bits."""
    y = torch.ones(n + offset, dtype=BF, device=DEV)[offset:]
    m.mhc_dropout(y, y, rng_state(), p=0.25, sequence=3)
    for at in (0, (1 << 30) - 7, LIMIT - 2050, (1 << 32) - 2050, (1 << 33) - 2050, (1 << 34) - 2050, (1 << 34) + 95000, n - 4099):
        if 0 <= at < n:
            _check_dropout(y, 1.0, at, 0.25, 3)


@pytest.mark.parametrize("D", [2056, 2051])
def test_embedding(D):
    """A table and streams of more than 2^31 elements; the gradient of whole
    numbers is exact."""
    V, T = LIMIT // D + 300, LIMIT // (4 * D) + 300
    g = torch.Generator(device=DEV).manual_seed(1)
    ids = torch.randint(0, V, (T,), generator=g, device=DEV)
    ids[-40:] = torch.arange(V - 40, V, device=DEV)   # the table's last rows
    ids[:20] = V - 3
    table = torch.empty(V, D, dtype=BF, device=DEV)
    table[:] = torch.arange(V, device=DEV)[:, None] % 251
    table += (torch.arange(D, device=DEV) % 5).to(BF)
    x = torch.empty(T, 4 * D, dtype=BF, device=DEV)
    m.mhc_embed_forward(ids, table, x)
    want = ids[:, None] % 251 + torch.arange(D, device=DEV) % 5
    for s in range(4):
        assert torch.equal(x[:, s * D:(s + 1) * D], want.to(BF))   # at most 255: exact in BF16
    del table
    got = torch.empty(V, D, device=DEV)
    m.mhc_embed_backward(ids, x, got, scratch(m.mhc_embed_workspace_bytes(T, V, D)))
    count = torch.bincount(ids, minlength=V)
    row = torch.arange(V, device=DEV)
    for lo in range(0, V, 100000):
        hi = min(V, lo + 100000)
        expected = 4 * count[lo:hi, None] * (row[lo:hi, None] % 251 + torch.arange(D, device=DEV) % 5)
        assert torch.equal(got[lo:hi], expected.float())
