"""Layer norms whose operands are column slices of one buffer: the results are
those of separate tensors, bit for bit, and no other column changes."""
import pytest
import torch

import rms_backward_gb300 as m

from operators_cases import DEV, DTYPES, empty, gen, normal, scratch

pytestmark = pytest.mark.gpu


def _slices(T, D, dtype, count, gap, *values):
    """`count` slices of D columns, `gap` columns apart, the first ones holding
    `values`, the others NaN; and the buffer."""
    buffer = torch.full((T, count * (D + gap) + 8 + gap % 2), float("nan"), dtype=dtype, device=DEV)
    parts = [buffer[:, k * (D + gap):k * (D + gap) + D] for k in range(count)]
    for part, v in zip(parts, values):
        part.copy_(v)
    return buffer, parts


# in registers, through shared memory, read again; rows on 16-byte boundaries where D + gap is a multiple of 8
@pytest.mark.parametrize("T,D,gap", [(5, 7, 0), (5, 7, 6), (5, 64, 0), (5, 64, 7), (700, 1285, 0), (700, 1285, 1),
                                     (700, 1280, 31), (700, 1280, 8), (3, 5121, 2), (400, 5120, 7), (400, 5120, 0),
                                     (2, 20481, 0), (2, 20480, 0), (200, 12289, 1), (200, 12288, 8)])
@pytest.mark.parametrize("type_", ["bf16", "fp16", "fp32"])
def test_norm_in_slices_of_one_buffer(T, D, gap, type_):
    g, dt = gen(T + D), DTYPES[type_]
    x, gy = normal(g, T, D, dtype=dt).to(DEV), normal(g, T, D, dtype=dt).to(DEV)
    gamma, beta = normal(g, D).to(DEV), normal(g, D).to(DEV)

    def both(x, y, gy, gx):
        mean, rstd, gg, gb = empty(T), empty(T), empty(D), empty(D)
        m.mhc_layernorm_forward(x, gamma, beta, y, mean, rstd)
        m.mhc_layernorm_backward(x, gy, gamma, mean, rstd, gx, gg, gb, scratch(m.mhc_layernorm_workspace_bytes(T, D)))
        return mean, rstd, gg, gb

    buffer, (bx, by, bgy, bgx) = _slices(T, D, dt, 4, gap, x, x, gy, gy)
    by.fill_(float("nan"))
    bgx.fill_(float("nan"))
    # the same distances between rows and to 16-byte boundaries, in buffers of their own
    apart = []
    for k, v in enumerate((x, None, gy, None)):
        _, parts = _slices(T, D, dt, 4, gap)
        if v is not None:
            parts[k].copy_(v)
        apart.append(parts[k])
    got, want = both(bx, by, bgy, bgx), both(*apart)
    for a, b in zip((by, bgx, *got), (apart[1], apart[3], *want)):
        assert torch.equal(a, b) and bool(torch.isfinite(a).all())
    assert torch.equal(bx, x) and torch.equal(bgy, gy)
    for k in range(4):
        assert bool(torch.isnan(buffer[:, k * (D + gap) + D:(k + 1) * (D + gap)]).all())
    assert bool(torch.isnan(buffer[:, 4 * (D + gap):]).all())
