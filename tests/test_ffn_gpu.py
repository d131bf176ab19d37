"""The gated feed-forward block and its gradient on the GPU against the FP64
oracle: elementwise bounds, and whole numbers to the last bit, over both shapes
of the product kernel, tile borders, odd sizes, row strides and few tokens."""
import pytest
import torch

import oracle.mhcm_oracle as O
import rms_backward_gb300 as m
from rms_backward_gb300 import abi

import matrix_cases as M
from matrix_cases import DEV, f64

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16

SMALL = [(8, 1024, 2560), (48, 520, 3000), (7, 264, 5000), (64, 72, 136), (65, 72, 136), (3, 75, 141), (4, 1001, 77), (2, 2048, 4096), (1, 1027, 515), (1, 1, 1), (1, 8, 8), (1, 64, 64), (2, 7, 3), (1, 136, 1000), (5, 1000, 136), (8, 2048, 72), (64, 256, 512),
         (1, 5003, 2309), (2, 2309, 4501), (4, 1286, 1284),
         (127, 129, 131), (128, 128, 128), (129, 320, 257), (257, 200, 264), (300, 65, 700)]
# tiles of 256 x 256 in every product, in some, odd ones
LARGE = [(1100, 1601, 1600), (300, 2600, 2568), (2049, 136, 2500), (700, 1032, 3432)]


@pytest.mark.parametrize("T,D,F", SMALL)
@pytest.mark.parametrize("type_,act", [("bf16", "silu"), ("fp16", "gelu")])
def test_forward(T, D, F, type_, act):
    M.ffn_forward_case(T, D, F, type_, act, seed=T + D + F)


@pytest.mark.parametrize("T,D,F", SMALL)
@pytest.mark.parametrize("type_,act,grad_type", [("bf16", "silu", "bf16"), ("bf16", "gelu", "fp32"), ("fp16", "silu", "fp16")])
def test_backward(T, D, F, type_, act, grad_type):
    M.ffn_backward_case(T, D, F, type_, act, grad_type, seed=T + D + F)


@pytest.mark.parametrize("T,D,F", SMALL + LARGE)
@pytest.mark.parametrize("type_,grad_type", [("bf16", "fp32"), ("fp16", "fp16")])
def test_whole_numbers(T, D, F, type_, grad_type):
    M.ffn_exact_case(T, D, F, type_, seed=T + D + F, grad_type=grad_type)


@pytest.mark.parametrize("T,D,F", LARGE)
def test_large(T, D, F):
    M.ffn_forward_case(T, D, F, "bf16", "silu", seed=1)
    M.ffn_backward_case(T, D, F, "bf16", "silu", seed=1)


@pytest.mark.parametrize("T,D,F", [(40, 72, 200), (600, 1048, 2056)])
@pytest.mark.parametrize("pad", [8, 64])
def test_row_strides(T, D, F, pad):
    M.ffn_forward_case(T, D, F, "bf16", pad=pad, seed=pad)
    M.ffn_backward_case(T, D, F, "bf16", pad=pad, seed=pad)


@pytest.mark.parametrize("T,D,F", [(40, 72, 200), (33, 75, 141), (600, 1040, 2056)])
@pytest.mark.parametrize("type_,grad_type", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp32")])
def test_added_gradients(T, D, F, type_, grad_type):
    M.ffn_backward_case(T, D, F, type_, grad_type=grad_type, accumulate=True, seed=9)


@pytest.mark.parametrize("which", [(1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 1, 0), (0, 0, 0, 1), (1, 1, 1, 0), (0, 1, 1, 1)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_outputs_left_out(which, accumulate):
    M.ffn_backward_case(40, 72, 200, "bf16", which=which, accumulate=accumulate, seed=3)
    M.ffn_backward_case(21, 75, 141, "bf16", which=which, accumulate=accumulate, seed=3)


@pytest.mark.parametrize("T", [1, 4, 5, 40, 64])
def test_few_tokens_lose_nothing_between_the_products(T):
    """Up to 64 tokens the forward's and grad_x's only rounding to 16 bits is the output's: with few
    elements the ones between the products would not average out.  (FP32 sums and the 16 bits that are
    kept of a, dg and du: below 2^-13 of the result in the 2-norm.)"""
    D, F = 72, 264
    _, x, wg, wu, wd = M.inputs(T, D, F, BF, T)
    y = torch.empty_like(x)
    gate, up = (torch.empty(T, F, dtype=BF, device=DEV) for _ in range(2))
    ws, _ = M.scratch(max(m.mhc_ffn_forward_workspace_bytes(T, D, F), m.mhc_ffn_backward_workspace_bytes(T, D, F)))
    m.mhc_ffn_forward(x, wg, wu, wd, y, ws, gate, up)
    m.mhc_ffn_backward(x, wg, wu, wd, gate, up, x, dx := torch.empty_like(x), None, None, None, ws)
    inputs = list(map(f64, (x, wg, wu, wd)))
    ref = [O.ffn_forward(*inputs, "silu", "bf16")[0][0], O.ffn_backward(*inputs, f64(gate), f64(up), inputs[0], "silu", "bf16", "bf16")[0][0]]
    for got, r in zip((y, dx), ref):
        once = torch.from_numpy(r).float().to(BF).double().numpy()
        assert abs(f64(got) - r).max() <= (2.0 ** -8 + 2.0 ** -11) * abs(r).max()
        assert ((f64(got) - r) ** 2).sum() ** 0.5 <= ((once - r) ** 2).sum() ** 0.5 + 2.0 ** -13 * (r ** 2).sum() ** 0.5


def test_no_outputs_and_no_tokens():
    x, w, wd = (torch.ones(s, dtype=BF, device=DEV) for s in ((0, 16), (24, 16), (16, 24)))
    t = torch.empty(0, 24, dtype=BF, device=DEV)
    ws = torch.empty(0, dtype=torch.uint8, device=DEV)
    m.mhc_ffn_forward(x, w, w, wd, torch.empty_like(x), ws)
    grads = [torch.full_like(v, 3.0) for v in (w, w, wd)]
    m.mhc_ffn_backward(x, w, w, wd, t, t, x, torch.empty_like(x), *grads, ws, accumulate=True)
    assert all((g == 3).all() for g in grads)
    m.mhc_ffn_backward(x, w, w, wd, t, t, x, None, grads[0], None, grads[2], ws)
    assert (grads[0] == 0).all() and (grads[1] == 3).all() and (grads[2] == 0).all()
    m.mhc_ffn_backward(x, w, w, wd, t, t, x, None, None, None, None, None)


@pytest.mark.parametrize("T,D,F", [(1, 1024, 2560), (48, 520, 1304), (300, 1032, 2600), (1000, 257, 515)])
def test_same_bits_again(T, D, F):
    """Every call gives the same bits, whatever the workspace and the outputs held."""
    a = M.ffn_forward_case(T, D, F, "bf16", seed=5)
    b = M.ffn_forward_case(T, D, F, "bf16", seed=5)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    # the backward twice on one set of buffers
    x, wg, wu, wd, y, gate, up = a
    outs = []
    for fill in (0x00, 0x7F):
        grads = [torch.empty_like(t) for t in (x, wg, wu, wd)]
        ws = torch.full((m.mhc_ffn_backward_workspace_bytes(T, D, F),), fill, dtype=torch.uint8, device=DEV)
        m.mhc_ffn_backward(x, wg, wu, wd, gate, up, y, *grads, ws)
        outs.append(grads)
    assert all(torch.equal(p, q) for p, q in zip(*outs))


@pytest.mark.parametrize("T", [3, 200])
def test_a_token_keeps_its_non_finite_values(T):
    """NaN and infinity in one token reach that token's rows and the weights' gradients only."""
    D, F = 136, 264
    _, x, wg, wu, wd = M.inputs(T, D, F, BF, 4)
    clean = [torch.empty(T, n, dtype=BF, device=DEV) for n in (D, F, F)]
    ws, _ = M.scratch(m.mhc_ffn_forward_workspace_bytes(T, D, F))
    m.mhc_ffn_forward(x, wg, wu, wd, clean[0], ws, *clean[1:])
    bad = x.clone()
    bad[1, 5], bad[2, 7] = float("nan"), float("inf")
    got = [torch.empty_like(t) for t in clean]
    m.mhc_ffn_forward(bad, wg, wu, wd, got[0], ws, *got[1:])
    keep = [t for t in range(T) if t not in (1, 2)]
    for p, q in zip(clean, got):
        assert torch.equal(p[keep], q[keep]) and not torch.isfinite(q[1]).any()
        assert not torch.isfinite(q[2]).all()


@pytest.mark.parametrize("T,D,F", [(1, 1027, 515), (2, 75, 141), (4, 139, 77), (1, 136, 264), (70, 75, 141)])
def test_a_row_of_weights_keeps_its_non_finite_values(T, D, F):
    """NaN in some rows of the weights reaches those rows' products only: rows that share 16 bytes do not mix."""
    _, x, wg, wu, wd = M.inputs(T, D, F, BF, 6)
    ws, _ = M.scratch(m.mhc_ffn_forward_workspace_bytes(T, D, F))
    clean = [torch.empty(T, n, dtype=BF, device=DEV) for n in (D, F, F)]
    m.mhc_ffn_forward(x, wg, wu, wd, clean[0], ws, *clean[1:])
    got = [torch.empty_like(t) for t in clean]
    gates, downs = [0, 2, F // 2, F - 1], [1, D // 3, D - 2]
    bad = wd.clone()
    bad[downs] = float("nan")
    m.mhc_ffn_forward(x, wg, wu, bad, got[0], ws, *got[1:])
    keep = [i for i in range(D) if i not in downs]
    assert torch.equal(got[0][:, keep], clean[0][:, keep]) and got[0][:, downs].isnan().all()
    bad, up = wg.clone(), wu.clone()
    bad[gates], up[gates] = float("nan"), float("inf")
    m.mhc_ffn_forward(x, bad, up, wd, got[0], ws, *got[1:])
    keep = [i for i in range(F) if i not in gates]
    assert all(torch.equal(q[:, keep], c[:, keep]) and not q[:, gates].isfinite().any()
               for q, c in zip(got[1:], clean[1:]))


def test_large_gates():
    """Gates far out on both sides, and zeros: no overflow inside the activation."""
    T, F, D = 4, 64, 64
    g = torch.Generator().manual_seed(1)
    gate = torch.tensor([-3e38, -1e4, -200., -88., -40., -9., -1e-30, 0., 1e-30, 9., 40., 88., 200., 1e4, 1e19, 1e-39])
    gate = gate.repeat(T, F // 16).to(BF).to(DEV)
    up, dy = (torch.randn(T, n, generator=g).to(BF).to(DEV) for n in (F, D))
    wd = torch.eye(D, F).to(BF).to(DEV)
    x = torch.randn(T, D, generator=g).to(BF).to(DEV)
    for act in ("silu", "gelu"):
        grads = [torch.empty(F, D, device=DEV), torch.empty(F, D, device=DEV), torch.empty(D, F, device=DEV)]
        ws, _ = M.scratch(m.mhc_ffn_backward_workspace_bytes(T, D, F))
        m.mhc_ffn_backward(x, wd, wd, wd, gate, up, dy, None, *grads, ws, activation=act)
        ref, bound = O.ffn_backward(*map(f64, (x, wd, wd, wd, gate, up, dy)), act, "bf16", "fp32")
        for got, r, b in zip(grads, ref[1:], bound[1:]):
            M.within(act, got, r, b)


def test_device_wait_that_runs_out():
    """A wait that nothing ends is given up after its limit and reported; later calls are sound."""
    T, D, F = 64, 64, 64
    t = [torch.zeros(64, 64, dtype=BF, device=DEV) for _ in range(12)]
    size = m.mhc_ffn_backward_workspace_bytes(T, D, F)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    p = [v.data_ptr() for v in t]
    stream = torch.cuda.current_stream().cuda_stream
    assert m.mhc_operators_device_status() == abi.MHCPB_OK
    abi.mhcpb_ffn_backward(T, D, F, abi.MHCPB_BF16, abi.MHCPB_SILU, p[0], D, *p[1:6], p[6], D, p[7], D, abi.MHCPB_BF16,
                           *p[8:11], abi.MHCPB_TEST_INJECT_STALL, ws.data_ptr(), size, stream)
    assert m.mhc_operators_device_status(clear=True) == abi.MHCPB_ERR_DEVICE_TIMEOUT
    assert m.mhc_operators_device_status() == abi.MHCPB_OK
    M.ffn_backward_case(T, D, F, "bf16", seed=2)
    assert m.mhc_operators_device_status() == abi.MHCPB_OK
