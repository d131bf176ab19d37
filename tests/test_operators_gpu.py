"""GPU parity of the operators around the stage (include/mhcpb.h) with the
FP64 oracle, at the sizes where they can go wrong: no token, one token, one
column, odd and unaligned rows, rows too long for registers, tables larger and
smaller than the batch, one id for most tokens, more tokens than one sorted
tile.  The bounds are those of oracle/mhcs_oracle.py with the chains derived
in operators_cases.py."""
import numpy as np
import pytest
import torch

import oracle.mhcs_oracle as S
import rms_backward_gb300 as m

import operators_cases as C
from operators_cases import DEV, empty, gen, normal, np64, rng_state, scratch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


# ---------------------------------------------------------------- embedding
@pytest.mark.parametrize("T,V,D,n", [(1, 1, 1, 1), (3, 50, 5120, 4), (77, 9, 1285, 4), (40, 300, 40, 16),
                                     (129, 1000, 24, 2), (5, 7, 4097, 1)])
@pytest.mark.parametrize("type_,wide", [("bf16", True), ("fp16", False), ("fp32", True)])
def test_embed_forward(T, V, D, n, type_, wide):
    C.embed_forward_case(T, V, D, n, type_, wide, seed=T + D)


@pytest.mark.parametrize("T,V,D,n", [(1, 1, 1, 1), (1, 70, 8, 4), (31, 33, 72, 4), (33, 5, 1285, 1), (500, 2000, 40, 4),
                                     (4096, 37, 16, 2), (4097, 5000, 8, 1), (9001, 64, 3, 4), (70000, 900, 8, 1),
                                     (16385, 100000, 8, 1), (300000, 5000, 1, 1)])   # one, two and three merges
@pytest.mark.parametrize("wide,accumulate", [(True, False), (False, True)])
def test_embed_backward(T, V, D, n, wide, accumulate):
    C.embed_backward_case(T, V, D, n, wide, accumulate, seed=T + D)


@pytest.mark.parametrize("T,V,D", [(200, 3, 24), (5000, 401, 17), (40000, 64, 8)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embed_backward_one_frequent_id(T, V, D, accumulate):
    """A run that crosses many chunks (and, above 4096 tokens, sorted tiles)."""
    C.embed_backward_case(T, V, D, 4, True, accumulate, seed=T, skew=True)


@pytest.mark.parametrize("D", [8, 40, 1031, 1032, 2056])
@pytest.mark.parametrize("offset", [1, 2, 5])
def test_embed_unaligned(D, offset):
    """Tensors that start anywhere: rows begin and end inside 16-byte chunks."""
    C.embed_forward_case(37, 50, D, 3, "fp32", True, seed=D, offset=offset)
    C.embed_forward_case(37, 50, D, 4, "bf16", False, seed=D, offset=offset)
    C.embed_backward_case(300, 41, D, 4, True, False, seed=D, offset=offset)
    C.embed_backward_case(300, 41, D, 1, False, True, seed=D, offset=offset, skew=True)


@pytest.mark.parametrize("D", [1, 2, 3, 5, 7, 9, 11, 13])
def test_embed_rows_shorter_than_a_vector(D):
    C.embed_forward_case(700, 30, D, 4, "bf16", True, seed=D)
    C.embed_backward_case(700, 30, D, 4, True, False, seed=D)
    C.embed_backward_case(700, 30, D, 2, True, True, seed=D)


def test_embed_backward_same_bits():
    g = gen(5)
    T, V, D = 9000, 50, 264
    ids = torch.randint(0, V, (T,), generator=g).to(DEV)
    gx = normal(g, T, 4 * D, dtype=BF).to(DEV)
    ws = scratch(m.mhc_embed_workspace_bytes(T, V, D))
    outs = []
    for _ in range(3):
        out = empty(V, D)
        m.mhc_embed_backward(ids, gx, out, ws)
        outs.append(out)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_embed_no_tokens():
    ids = torch.empty(0, dtype=torch.int64, device=DEV)
    x = torch.empty(0, 32, dtype=BF, device=DEV)
    table, ws = torch.ones(5, 8, device=DEV), torch.empty(0, dtype=torch.uint8, device=DEV)
    m.mhc_embed_forward(ids, table, x)
    assert m.mhc_embed_workspace_bytes(0, 5, 8) == 0
    m.mhc_embed_backward(ids, x, table, ws, accumulate=True)
    assert bool((table == 1).all())
    m.mhc_embed_backward(ids, x, table, ws)
    assert not table.any()


def test_embed_extreme_ids():
    """Ids whose low 32 bits look valid are still outside the table."""
    ids = torch.tensor([2**32 + 1, -2**63, 2**63 - 1, 1, -1, 3], device=DEV)
    table = torch.arange(1.0, 4.0, device=DEV)[:, None].expand(3, 8).contiguous()
    x = empty(6, 8, dtype=BF)
    m.mhc_embed_forward(ids, table, x)
    assert x[:, 0].tolist() == [0, 0, 0, 2, 0, 0]
    g = empty(3, 8)
    m.mhc_embed_backward(ids, torch.ones(6, 8, dtype=BF, device=DEV), g, scratch(m.mhc_embed_workspace_bytes(6, 3, 8)))
    assert g[:, 0].tolist() == [0, 1, 0]


# ---------------------------------------------------------------- layer norm
NORM_SHAPES = [(1, 1), (1, 5120), (3, 2), (5, 7), (33, 40), (300, 128), (17, 1285), (9, 8200), (2, 20000), (3, 70001),
               (700, 64), (2, 131072)]


@pytest.mark.parametrize("T,D", NORM_SHAPES)
@pytest.mark.parametrize("type_", ["bf16", "fp16", "fp32"])
def test_norm_forward(T, D, type_):
    C.norm_forward_case(T, D, type_, seed=T + D, eps=1e-5)


@pytest.mark.parametrize("T,D", NORM_SHAPES)
@pytest.mark.parametrize("type_", ["bf16", "fp16", "fp32"])
def test_norm_backward(T, D, type_):
    C.norm_backward_case(T, D, type_, seed=T + D)


@pytest.mark.parametrize("type_,D,pad", [("bf16", 40, 8), ("bf16", 40, 1), ("fp32", 37, 3), ("fp16", 5120, 8), ("fp32", 64, 4)])
def test_norm_row_strides(type_, D, pad):
    C.norm_forward_case(19, D, type_, seed=D, pad=pad)
    C.norm_backward_case(19, D, type_, seed=D, pad=pad)


def test_norm_without_parameters_or_statistics():
    C.norm_forward_case(10, 48, "bf16", seed=1, affine=False, stats=False)
    C.norm_forward_case(10, 47, "fp32", seed=1, affine=False)
    for params in ("none", "beta"):
        C.norm_backward_case(10, 48, "bf16", seed=2, affine=False, params=params)
        C.norm_backward_case(10, 47, "fp32", seed=2, params=params)


@pytest.mark.parametrize("T,D", [(0, 24), (1, 24), (900, 24), (900, 25)])
def test_norm_backward_accumulates(T, D):
    C.norm_backward_case(T, D, "bf16", seed=3, accumulate=True)


def test_norm_no_tokens():
    x = torch.empty(0, 24, device=DEV)
    m.mhc_layernorm_forward(x, None, None, x.clone())
    gg, gb = empty(24), empty(24)
    e = torch.empty(0, device=DEV)
    m.mhc_layernorm_backward(x, x.clone(), None, e, e.clone(), x.clone(), gg, gb)
    assert not gg.any() and not gb.any()


def test_norm_large_offset():
    """Rows far from zero: the variance is centred, so nothing cancels.  Against
    the same FP32 values in FP64 (a mean of squares would lose every digit)."""
    g = gen(8)
    x = (1000.0 + normal(g, 7, 515)).to(DEV)
    y, mean, rstd = empty(7, 515), empty(7), empty(7)
    m.mhc_layernorm_forward(x, None, None, y, mean, rstd)
    _, _, want, *_ = S.norm_forward(np64(x), 1.0, 0.0, 1e-5)
    # var's relative error: (error of the mean)^2 <= (chain 2^-24 1000)^2 ~ 2.3e-5 at chain 80, and the chain itself
    assert np.all(np.abs(np64(rstd) / want - 1) <= 80 * 2.0**-24 + (80 * 2.0**-24 * 1000) ** 2)


def test_norm_nan_stays_in_its_row():
    x = normal(gen(9), 8, 136, dtype=BF).to(DEV)
    x[3, 5] = float("nan")
    x[6, 7] = float("inf")
    y = empty(8, 136, dtype=BF)
    m.mhc_layernorm_forward(x, None, None, y)
    bad = torch.isnan(y).all(1).tolist()
    assert bad == [False, False, False, True, False, False, True, False] and torch.isnan(y).sum() == 2 * 136


def test_norm_forward_gradient_by_differences():
    """Central differences of the FP32 forward along a direction against
    <grad_x, direction>: truncation O(eps^2) plus forward rounding of about
    2^-24 sqrt(elements) / eps, both under 1e-3 of the sum's scale here."""
    g = gen(10)
    T, D = 6, 96
    x, v, gy, gamma = (normal(g, *s).to(DEV) for s in ((T, D), (T, D), (T, D), (D,)))
    y, mean, rstd, gx = empty(T, D), empty(T), empty(T), empty(T, D)

    def value(a):
        m.mhc_layernorm_forward(a, gamma, None, y, mean, rstd)
        return (y.double() * gy.double()).sum().item()

    eps = 2.0**-8
    slope = (value(x + eps * v) - value(x - eps * v)) / (2 * eps)
    value(x)
    m.mhc_layernorm_backward(x, gy, gamma, mean, rstd, gx)
    want = (gx.double() * v.double()).sum().item()
    assert abs(slope - want) <= 1e-3 * (gx.double() * v.double()).abs().sum().item()


# ---------------------------------------------------------------- dropout
@pytest.mark.parametrize("shape,offset", [((1, 1), 0), ((3, 5), 0), ((64, 40), 0), ((7, 1285), 0), ((7, 1285), 1), ((2, 2056), 3)])
@pytest.mark.parametrize("type_", ["bf16", "fp16", "fp32"])
def test_dropout(shape, offset, type_):
    for p in (0.1, 0.5, 0.999):
        C.dropout_case(shape, type_, p, seed=shape[1], offset=offset)
    C.dropout_case(shape, type_, 0.3, seed=shape[1], in_place=True, offset=offset)


def test_dropout_drops_non_finite_values_and_p_zero_copies():
    x = torch.full((64, 64), float("nan"), device=DEV)
    y = empty(64, 64)
    m.mhc_dropout(x, y, rng_state(), p=0.5, sequence=9)
    keep = S.keep_mask((64, 64), 0.5, C.RNG, 9)
    assert np.array_equal(np.isnan(np64(y)), keep) and not np64(y)[~keep].any()
    v = normal(gen(1), 65, dtype=BF).to(DEV)
    out = empty(65, dtype=BF)
    m.mhc_dropout(v, out, p=0.0)
    assert torch.equal(out, v)


def test_dropout_graph_draws_new_masks():
    """A captured call reads the state when it runs: advancing the step between
    replays gives the masks of the uncaptured calls."""
    x, y = torch.ones(1000, device=DEV), empty(1000)
    state = rng_state()
    m.mhc_dropout(x, y, state, p=0.5)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mhc_dropout(x, y, state, p=0.5)
    seen = []
    for step in (3, 4):
        state[1] = step
        graph.replay()
        torch.cuda.synchronize()
        seen.append(y != 0)
        assert np.array_equal(seen[-1].cpu().numpy(), S.keep_mask((1000,), 0.5, (C.RNG[0], step)))
    assert not torch.equal(*seen)


# ---------------------------------------------------------------- collapse, update
STREAM_SHAPES = [(1, 1), (1, 5120), (2, 3), (5, 8), (33, 41), (70, 320), (9, 1285), (3, 8200), (2, 33000), (400, 72)]


@pytest.mark.parametrize("T,D", STREAM_SHAPES)
def test_collapse_norm(T, D):
    C.collapse_case(T, D, seed=T + D)


@pytest.mark.parametrize("D", [40, 41])
def test_collapse_norm_options(D):
    C.collapse_case(20, D, seed=1, residual=False)
    C.collapse_case(20, D, seed=2, params=False, affine=False)
    C.collapse_case(20, D, seed=3, accumulate=True)


@pytest.mark.parametrize("T,D", STREAM_SHAPES)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_update(T, D, p):
    C.update_case(T, D, p, seed=T + D)


@pytest.mark.parametrize("D", [40, 41])
def test_update_in_place(D):
    C.update_case(37, D, 0.25, seed=2, in_place=True)


# every number of warps per row and of rows per block that the hidden size can lead to
GROUP_SIZES = [8, 16, 32, 64, 104, 256, 264, 320, 512, 520, 640, 1024, 1280, 1288, 2560, 2568, 5120, 5128, 8192, 10240,
               10248]


@pytest.mark.parametrize("D", GROUP_SIZES)
def test_group_shapes(D):
    T = min(2400, 3_000_000 // D)
    C.norm_forward_case(T, D, "bf16", seed=D)
    C.norm_backward_case(T, D, "bf16", seed=D)
    C.collapse_case(T, D, seed=D)
    C.update_case(T, D, 0.0, seed=D)
    if D <= 10240 // 2:
        C.norm_forward_case(T, D, "fp32", seed=D)
        C.norm_backward_case(T, D, "fp32", seed=D)


@pytest.mark.parametrize("D", [9, 15, 31, 33, 127, 255, 257, 511, 1281, 2049, 2561, 4095, 4097, 5119, 8191, 8193])
def test_group_shapes_unaligned(D):
    T = min(2400, 2_000_000 // D)
    C.norm_forward_case(T, D, "bf16", seed=D)
    C.norm_backward_case(T, D, "fp32", seed=D)
    C.collapse_case(T, D, seed=D)
    C.update_case(T, D, 0.0, seed=D)


def test_streams_no_tokens():
    x, y, h = torch.empty(0, 32, dtype=BF, device=DEV), torch.empty(0, 8, dtype=BF, device=DEV), torch.empty(0, 24, device=DEV)
    e, gg, gb = torch.empty(0, device=DEV), empty(8), empty(8)
    m.mhc_update_forward(x, y, h, x.clone())
    m.mhc_update_backward(x, y, h, x.clone(), y.clone(), h.clone())
    m.mhc_collapse_norm_forward(x, h, None, None, y.clone())
    m.mhc_collapse_norm_backward(x, h, y, None, e, e.clone(), x.clone(), h.clone(), gg, gb)
    assert not gg.any() and not gb.any()


def test_update_masks_match_dropout():
    """The update draws the mask mhc_dropout draws for y: with H_res = 0 and
    H_post = 1 every stream is dropout(y)."""
    T, D = 13, 203
    g = gen(3)
    x, y = normal(g, T, 4 * D, dtype=BF).to(DEV), normal(g, T, D, dtype=BF).to(DEV)
    h = torch.zeros(T, 24, device=DEV)
    h[:, 4:8] = 1.0
    out, d = empty(T, 4 * D, dtype=BF), empty(T, D, dtype=BF)
    m.mhc_update_forward(x, y, h, out, rng_state(), p=0.4, sequence=2)
    m.mhc_dropout(y, d, rng_state(), p=0.4, sequence=2)
    for s in range(4):
        assert torch.equal(out[:, s * D:(s + 1) * D], d)


def test_gradients_same_bits():
    T, D = 1000, 328
    g = gen(4)
    x, go = (normal(g, T, 4 * D, dtype=BF).to(DEV) for _ in range(2))
    y, h = normal(g, T, D, dtype=BF).to(DEV), C.gates(g, T).to(DEV)
    mean, rstd, gamma = normal(g, T).to(DEV), (normal(g, T).abs() + 0.5).to(DEV), normal(g, D).to(DEV)
    ws = scratch(m.mhc_collapse_norm_workspace_bytes(T, D))
    seen = []
    for _ in range(2):
        gx, gh, gy, gg, gb = empty(T, 4 * D, dtype=BF), empty(T, 24), empty(T, D, dtype=BF), empty(D), empty(D)
        m.mhc_update_backward(x, y, h, go, gy, gh, rng_state(), p=0.1)
        m.mhc_collapse_norm_backward(x, h, gy, gamma, mean, rstd, gx, gh, gg, gb, ws, grad_x_out=go)
        seen.append([gx, gh, gy, gg, gb])
    for a, b in zip(*seen):
        assert torch.equal(a, b)


def test_streams_are_respected():
    """Calls on a side stream run there: each waits for what the stream holds."""
    side = torch.cuda.Stream()
    x = torch.zeros(4096, 512, device=DEV)
    out = empty(4096, 512)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        x.fill_(2.0)
    m.mhc_dropout(x, out, p=0.0, stream=side)
    side.synchronize()
    assert bool((out == 2.0).all())


# ---------------------------------------------------------------- refusals
def test_refusals_write_nothing():
    from rms_backward_gb300 import abi
    T, D = 6, 8
    x, xo = torch.ones(T, 4 * D, dtype=BF, device=DEV), torch.full((T, 4 * D), 7.0, dtype=BF, device=DEV)
    y, h = torch.ones(T, D, dtype=BF, device=DEV), torch.ones(T, 24, device=DEV)
    mean, gg = torch.ones(T, device=DEV), torch.full((D,), 7.0, device=DEV)
    P = lambda t: t.data_ptr()  # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    host = torch.ones(T, 4 * D, dtype=BF)
    need = m.mhc_layernorm_workspace_bytes(T, D)
    ws = scratch(need)
    calls = [
        (abi.MHCPB_ERR_ALIASING, lambda: abi.mhcpb_update_forward(T - 1, D, P(x), P(y), P(h), 0.0, None, 0, P(x) + 16, st)),
        (abi.MHCPB_ERR_WRONG_DEVICE, lambda: abi.mhcpb_update_forward(T, D, P(host), P(y), P(h), 0.0, None, 0, P(xo), st)),
        (abi.MHCPB_ERR_MISALIGNED, lambda: abi.mhcpb_update_forward(T - 1, D, P(x) + 2, P(y), P(h), 0.0, None, 0, P(xo), st)),
        (abi.MHCPB_ERR_INVALID_ARG, lambda: abi.mhcpb_update_forward(T, D, P(x), P(y), P(h), 0.5, None, 0, P(xo), st)),
        (abi.MHCPB_ERR_INVALID_ARG, lambda: abi.mhcpb_update_forward(T, D, P(x), P(y), P(h), 1.0, P(ws), 0, P(xo), st)),
        (abi.MHCPB_ERR_ALIASING, lambda: abi.mhcpb_update_backward(T, D, P(x), P(y), P(h), 0.0, None, 0, P(xo), P(y), P(h), st)),
        (abi.MHCPB_ERR_ALIASING, lambda: abi.mhcpb_dropout(T * D, 0, P(xo), 0.0, None, 0, P(xo) + 2, st)),
        (abi.MHCPB_ERR_INVALID_ARG, lambda: abi.mhcpb_dropout(T * D, 0, 0, 0.0, None, 0, P(xo), st)),
        (abi.MHCPB_ERR_WORKSPACE_TOO_SMALL, lambda: abi.mhcpb_layernorm_backward(
            T, D, 0, P(y), D, P(y), D, None, P(mean), P(mean), P(xo), D, P(gg), None, 0, P(ws), need - 1, st)),
        (abi.MHCPB_ERR_INVALID_ARG, lambda: abi.mhcpb_layernorm_forward(T, D, 0, P(y), D, None, None, 1e-5, P(xo), D,
                                                                        P(mean), None, st)),
        (abi.MHCPB_ERR_ALIASING, lambda: abi.mhcpb_collapse_norm_forward(T, D, P(x), P(h), P(gg), None, 1e-5, P(xo),
                                                                         P(gg), P(mean), st)),
        (abi.MHCPB_ERR_WRONG_DEVICE, lambda: abi.mhcpb_embed_forward(T, T, D, 4, 0, P(host), P(x), 8, 1.0, P(xo), st)),
        (abi.MHCPB_ERR_MISALIGNED, lambda: abi.mhcpb_embed_forward(2, 2, D, 4, 0, P(y), P(x) + 4, 8, 1.0, P(xo), st)),
    ]
    for status, call in calls:
        with pytest.raises(abi.MhcpbError) as e:
            call()
        assert e.value.status == status, (status, e.value)
    torch.cuda.synchronize()
    assert bool((xo == 7).all()) and bool((gg == 7).all()) and bool((y == 1).all()) and bool((h == 1).all())
