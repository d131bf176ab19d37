"""The FP64 oracle of the operators around the stage, pinned on the CPU: the
generator to its published test vectors, every gradient to central differences
of its own forward, and planted mistakes to the acceptance check."""
import numpy as np
import pytest

import oracle.mhcs_oracle as S

RNG = (0x0123456789ABCDEF, 5)


@pytest.mark.parametrize("counter,key,want", [
    # known answers published with the generator (Random123, philox 4x32, 10 rounds)
    ([0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
    ([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
    ([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
     [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]),
])
def test_generator_known_answers(counter, key, want):
    assert S.philox(counter, key) == want


def test_words_follow_the_counter():
    words = S.random_words(11, RNG, sequence=7)
    key, step = RNG[0], RNG[1] + 7
    for e in range(11):
        c = S.philox((e // 4, 0, step, 0), (key & 0xFFFFFFFF, key >> 32))
        assert words[e] == c[e % 4]
    # the step and the sequence number enter as one sum, modulo 2^64
    assert np.array_equal(S.random_words(8, (3, 2**64 - 1), 1), S.random_words(8, (3, 0)))


def test_dropout_share_and_zero_probability():
    x = np.ones((64, 65))
    y = S.dropout(x, 0.25, RNG)
    assert set(np.unique(y)) == {0.0, S.keep_scale(0.25)}
    share = (y == 0).mean()
    assert abs(share - 0.25) < 5 * np.sqrt(0.25 * 0.75 / y.size)   # five standard deviations
    assert np.array_equal(S.dropout(x, 0.0, None), x)
    assert not np.array_equal(S.keep_mask(x.shape, 0.25, RNG), S.keep_mask(x.shape, 0.25, RNG, 1))


def _differences(f, a, weights, eps=1e-6):
    """d (sum weights * f) / da by central differences."""
    g = np.zeros_like(a)
    it = np.nditer(a, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = a[i]
        a[i] = keep + eps
        hi = (f() * weights).sum()
        a[i] = keep - eps
        lo = (f() * weights).sum()
        a[i] = keep
        g[i] = (hi - lo) / (2 * eps)
    return g


def test_norm_gradients_against_differences():
    r = np.random.default_rng(1)
    u, gamma, beta, gy = r.normal(size=(3, 7)), r.normal(size=7), r.normal(size=7), r.normal(size=(3, 7))
    f = lambda: S.norm_forward(u, gamma, beta, 1e-5)[0]  # noqa: E731
    _, mean, rstd, *_ = S.norm_forward(u, gamma, beta, 1e-5)
    (du, gg, gb), _ = S.norm_backward(u, gy, gamma, mean, rstd)
    for a, g in ((u, du), (gamma, gg), (beta, gb)):
        assert np.allclose(_differences(f, a, gy), g, rtol=1e-6, atol=1e-7)


def test_sublayer_gradients_against_differences():
    """X reaches the next streams through H_res and through the collapse; both
    gradients of X together, and those of the gates and of y, match."""
    r = np.random.default_rng(2)
    T, D = 2, 5
    x, h, y0 = r.normal(size=(T, 4 * D)), r.uniform(0.2, 1.0, size=(T, 24)), r.normal(size=(T, D))
    gamma, beta, go = r.normal(size=D), r.normal(size=D), r.normal(size=(T, 4 * D))
    p = 0.4

    def both():   # the sublayer is y0 * (its input)
        u, _ = S.collapse(x, h)
        return S.update_forward(x, y0 * S.norm_forward(u, gamma, beta, 1e-5)[0], h, p, RNG)[0]

    u, _ = S.collapse(x, h)
    n, mean, rstd, *_ = S.norm_forward(u, gamma, beta, 1e-5)
    (gy, gh_rest), _ = S.update_backward(x, y0 * n, h, go, p, RNG)
    (gx, gh_pre, gg, gb), _ = S.collapse_norm_backward(x, h, gy * y0, gamma, mean, rstd, go)
    for a, g in ((x, gx), (h, np.concatenate([gh_pre, gh_rest], 1)), (gamma, gg), (beta, gb), (y0, gy * n)):
        assert np.allclose(_differences(both, a, go), g, rtol=1e-6, atol=1e-7)


def test_embedding_gradient_against_differences():
    r = np.random.default_rng(3)
    ids = np.array([2, 0, -1, 2, 4, 2, 5])   # -1 and 5 lie outside the table
    table, go = r.normal(size=(5, 3)), r.normal(size=(7, 6))
    g, mag, chain = S.embed_backward(ids, go, 5, 3, 0.75)
    assert np.allclose(_differences(lambda: S.embed_forward(ids, table, 2, 0.75), table, go), g, atol=1e-8)
    assert not g[[1, 3]].any() and not mag[[1, 3]].any()
    assert chain[2, 0] == 3 * 2 + 4
    assert not S.embed_forward(ids, table, 2, 0.75)[[2, 6]].any()


def test_acceptance_check_catches_mistakes():
    r = np.random.default_rng(4)
    u, gy = r.normal(size=(6, 64)), r.normal(size=(6, 64))
    gamma = r.normal(size=64)
    _, mean, rstd, *_ = S.norm_forward(u, gamma, 0.0, 1e-5)
    (du, gg, gb), (dum, ggm, gbm) = S.norm_backward(u, gy, gamma, mean, rstd)
    assert S.within(du, du, dum, 64)[0]
    assert S.within(du.astype(np.float32), du, dum, 2)[0]
    w = gy * gamma
    z = (u - mean[:, None]) * rstd[:, None]
    no_mean = rstd[:, None] * (w - z * (w * z).mean(1, keepdims=True))
    biased = rstd[:, None] * (w - w.mean(1, keepdims=True) - z * (w * z).sum(1, keepdims=True) / 63)
    for wrong in (no_mean, biased, np.where(np.isfinite(du), du, 0) * np.nan):
        assert not S.within(wrong, du, dum, 64)[0]
    assert not S.within((gy[:-1] * z[:-1]).sum(0), gg, ggm, 64)[0]
    assert not S.within(gb[:-1], gb, gbm, 64)[0]   # another shape
