"""The range of what the feed-forward block keeps between its products with FP16 operands, at both ends."""
import pytest
import torch

import oracle.mhcm_oracle as O
import rms_backward_gb300 as m

import matrix_cases as M
from matrix_cases import f64

pytestmark = pytest.mark.gpu
FP = torch.float16
D, F = 72, 264


@pytest.mark.parametrize("type_", ["fp16", "bf16"])
@pytest.mark.parametrize("T", [2, 4, 5, 64, 65, 200])
def test_large_activations(T, type_):
    """One token whose act(g) u passes 65,504: right in BF16, and up to four tokens in FP16; from five on that
    token's outputs are not finite, and the others keep their bits."""
    dtype = M.TYPES[type_]
    g, x, wg, wu, wd = M.inputs(T, D, F, dtype, T)
    wd = wd * 2.0 ** -10
    ws, _ = M.scratch(m.mhc_ffn_forward_workspace_bytes(T, D, F))
    clean, y = torch.empty_like(x), torch.empty_like(x)
    m.mhc_ffn_forward(x, wg, wu, wd, clean, ws)
    large = x.clone()
    large[1] *= 512.0
    gate, up = (torch.empty(T, F, dtype=dtype, device=x.device) for _ in range(2))
    m.mhc_ffn_forward(large, wg, wu, wd, y, ws, gate, up)
    (ref, rg, ru), (bound, bg, bu) = O.ffn_forward(*map(f64, (large, wg, wu, wd)), "silu", type_)
    assert abs(ref).max() < 2 ** 15 and abs(rg * ru).max() > 2 ** 17
    M.within("gate", gate, rg, bg)
    M.within("up", up, ru, bu)
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(y[keep], clean[keep])
    if type_ == "bf16" or T <= 4:
        M.within("y", y, ref, bound)
    else:
        assert not torch.isfinite(y[1]).any()


@pytest.mark.parametrize("grad_type", ["fp16", "fp32"])
@pytest.mark.parametrize("T", [40, 100])
def test_small_gradients(T, grad_type):
    """dg and du below 2^-25 are zero in FP16 (up to 64 tokens not for grad_x); with grad_y scaled by a power of
    two every gradient is right."""
    g, x, wg, wu, wd = M.inputs(T, D, F, FP, T)
    gate, up = (M.put(torch.randn(T, F, generator=g), FP) for _ in range(2))
    dy = M.put(2.0 ** -6 * torch.randn(T, D, generator=g), FP)
    ws, _ = M.scratch(m.mhc_ffn_backward_workspace_bytes(T, D, F))

    def run(dy_, wd_):
        dx, grads = torch.empty_like(x), [torch.empty(w.shape, dtype=M.TYPES[grad_type], device=x.device) for w in (wg, wu, wd)]
        m.mhc_ffn_backward(x, wg, wu, wd_, gate, up, dy_, dx, *grads, ws)
        ref, bound = O.ffn_backward(*map(f64, (x, wg, wu, wd_, gate, up, dy_)), "silu", "fp16", grad_type)
        return (dx, *grads), ref, bound

    # grad_y and a down projection so small that dg and du fall below 2^-25
    tiny = wd * 2.0 ** -12
    tiny_dy = dy * 2.0 ** -10
    (dx, gg, gu, gd), ref, bound = run(tiny_dy, tiny)
    act, slope, _, _ = O._act(f64(gate), "silu")
    da = f64(tiny_dy) @ f64(tiny)
    assert max(abs(da * f64(up) * slope).max(), abs(da * act).max()) < 2.0 ** -25
    assert not gg.any() and not gu.any()
    M.within("grad_w_down", gd, ref[3], bound[3])
    if T <= 64:
        M.within("grad_x", dx, ref[0], bound[0])
    got, ref, bound = run(dy * 2.0 ** 10, tiny)
    for name, q, r, b in zip(("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down"), got, ref, bound):
        assert abs(r).max() > 2.0 ** -20
        M.within(name, q, r, b)
