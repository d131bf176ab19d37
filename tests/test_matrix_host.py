"""Host-side refusals of the feed-forward block and of the orthogonalised update:
shapes, types, flags, strides and overlaps before any CUDA call, and the Python
layer's checks (all without a GPU)."""
import ctypes
import os

import pytest
import torch

import rms_backward_gb300 as m
from rms_backward_gb300 import abi

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from rms_backward_gb300 import build
        build.build()
    return abi.load()


SHAPE, ARG, SMALL = abi.MHCPB_ERR_UNSUPPORTED_SHAPE, abi.MHCPB_ERR_INVALID_ARG, abi.MHCPB_ERR_WORKSPACE_TOO_SMALL
ALIGN, ALIAS = abi.MHCPB_ERR_MISALIGNED, abi.MHCPB_ERR_ALIASING
TOO_LONG, TOO_WIDE = (1 << 24) + 1, (1 << 20) + 1
BIG = 1 << 40   # workspace bytes that are enough for anything


def at(i):
    """Addresses far from one another; nothing reads them."""
    return (i + 1) << 44


def forward(T=4, D=16, F=24, type_=0, act=0, x=at(0), xs=None, wg=at(1), wu=at(2), wd=at(3), y=at(4), ys=None, gate=at(5),
            up=at(6), ws=at(7), size=BIG):
    return abi.mhcpb_ffn_forward(T, D, F, type_, act, x, D if xs is None else xs, wg, wu, wd, y, D if ys is None else ys,
                                 gate, up, ws, size, None)


def backward(T=4, D=16, F=24, type_=0, act=0, x=at(0), xs=None, wg=at(1), wu=at(2), wd=at(3), gate=at(4), up=at(5), dy=at(6),
             dys=None, dx=at(7), dxs=None, gtype=0, gg=at(8), gu=at(9), gd=at(10), flags=0, ws=at(11), size=BIG):
    return abi.mhcpb_ffn_backward(T, D, F, type_, act, x, D if xs is None else xs, wg, wu, wd, gate, up, dy,
                                  D if dys is None else dys, dx, D if dxs is None else dxs, gtype, gg, gu, gd, flags, ws, size,
                                  None)


def orth(mm=40, n=64, type_=2, g=at(0), gs=None, steps=5, eps=1e-7, scale=1.0, out=at(1), os_=None, ws=at(2), size=BIG):
    return abi.mhcpb_orthogonalize(mm, n, type_, g, n if gs is None else gs, steps, eps, scale, out,
                                   n if os_ is None else os_, ws, size, None)


@pytest.mark.parametrize("status,call,kw", [
    (SHAPE, forward, dict(T=-1)), (SHAPE, forward, dict(T=TOO_LONG)), (SHAPE, forward, dict(D=0)),
    (SHAPE, forward, dict(D=TOO_WIDE)), (SHAPE, forward, dict(F=0)), (SHAPE, forward, dict(F=TOO_WIDE)),
    (SHAPE, forward, dict(xs=15)), (SHAPE, forward, dict(xs=17)), (SHAPE, forward, dict(ys=20)), (SHAPE, forward, dict(ys=-16)),
    (SHAPE, forward, dict(xs=(1 << 24) + 8)),
    (ARG, forward, dict(type_=2)), (ARG, forward, dict(type_=-1)), (ARG, forward, dict(act=2)),
    (ARG, forward, dict(gate=None)), (ARG, forward, dict(up=None)), (ARG, forward, dict(x=None)), (ARG, forward, dict(wd=None)),
    (ARG, forward, dict(y=None)), (SMALL, forward, dict(size=0)),
    (ALIGN, forward, dict(x=at(0) + 8)), (ALIGN, forward, dict(wg=at(1) + 2)), (ALIGN, forward, dict(gate=at(5) + 4)),
    (ALIGN, forward, dict(ws=at(7) + 8)),
    (ALIAS, forward, dict(y=at(0))), (ALIAS, forward, dict(gate=at(1))), (ALIAS, forward, dict(up=at(5))),
    (ALIAS, forward, dict(ws=at(3))), (ALIAS, forward, dict(y=at(0) + 4 * 16 * 2 - 16)),
    (SHAPE, backward, dict(T=-3)), (SHAPE, backward, dict(D=TOO_WIDE)), (SHAPE, backward, dict(dys=9)),
    (SHAPE, backward, dict(dxs=17)), (ARG, backward, dict(type_=2, gtype=2)), (ARG, backward, dict(gtype=1)),
    (ARG, backward, dict(flags=1)), (ARG, backward, dict(gate=None)), (ARG, backward, dict(dy=None)),
    (SMALL, backward, dict(size=64)), (ALIGN, backward, dict(gd=at(10) + 4)), (ALIAS, backward, dict(dx=at(6))),
    (ALIAS, backward, dict(gg=at(9))), (ALIAS, backward, dict(gu=at(5))), (ALIAS, backward, dict(gd=at(3))),
    (ALIAS, backward, dict(gg=at(1), gtype=2)),
    (SHAPE, orth, dict(mm=0)), (SHAPE, orth, dict(n=0)), (SHAPE, orth, dict(mm=TOO_WIDE)), (SHAPE, orth, dict(n=TOO_WIDE)),
    (SHAPE, orth, dict(steps=0)), (SHAPE, orth, dict(steps=33)), (SHAPE, orth, dict(gs=63)), (SHAPE, orth, dict(os_=65)),
    (ARG, orth, dict(type_=3)), (ARG, orth, dict(eps=-1e-9)), (ARG, orth, dict(eps=float("nan"))),
    (ARG, orth, dict(eps=float("inf"))), (ARG, orth, dict(scale=float("nan"))), (ARG, orth, dict(scale=float("inf"))),
    (ARG, orth, dict(g=None)), (ARG, orth, dict(out=None)), (SMALL, orth, dict(size=100)),
    (ALIGN, orth, dict(g=at(0) + 4)), (ALIGN, orth, dict(out=at(1) + 8)), (ALIAS, orth, dict(out=at(0))),
    (ALIAS, orth, dict(ws=at(1))),
])
def test_refused_before_cuda(status, call, kw):
    with pytest.raises(abi.MhcpbError) as e:
        call(**kw)
    assert e.value.status == status


@pytest.mark.parametrize("call,kw", [
    (forward, dict(gate=None, up=None)), (forward, dict(xs=24, ys=32)), (forward, dict(wu=at(1))), (forward, dict(D=15, F=7)),
    (backward, dict(dx=None)), (backward, dict(gg=None, gu=None)), (backward, dict(gtype=2)),
    (backward, dict(flags=abi.MHCPB_ACCUMULATE_DW)), (orth, dict(mm=64, n=33)), (orth, dict(gs=72, os_=128)),
    (orth, dict(mm=24, ws=None, size=0)),
])
def test_allowed_calls_reach_the_device_check(call, kw):
    """Nothing but the addresses (which are nobody's) is wrong with these."""
    with pytest.raises(abi.MhcpbError) as e:
        call(**kw)
    assert e.value.status not in (SHAPE, ARG, SMALL, ALIGN, ALIAS)


def test_slices_of_one_buffer():
    """y may lie between x's rows; a gate that lies there is refused."""
    base, row = at(0), 64
    with pytest.raises(abi.MhcpbError) as e:
        forward(x=base, xs=row, y=base + 2 * 16, ys=row)
    assert e.value.status not in (SHAPE, ARG, ALIGN, ALIAS)
    with pytest.raises(abi.MhcpbError) as e:
        forward(x=base, xs=row, gate=base + 2 * 16)
    assert e.value.status == ALIAS


def test_nothing_to_compute_is_no_error(lib):
    backward(dx=None, gg=None, gu=None, gd=None, ws=None, size=0)


def test_workspace_sizes(lib):
    n = ctypes.c_size_t()
    for f in (lib.mhcpb_ffn_forward_workspace_bytes, lib.mhcpb_ffn_backward_workspace_bytes):
        assert f(4, 4, 4, None) == ARG and f(-1, 4, 4, ctypes.byref(n)) == SHAPE and f(4, 0, 4, ctypes.byref(n)) == SHAPE
        assert f(0, 4, 4, ctypes.byref(n)) == abi.MHCPB_OK and n.value == 0
    assert lib.mhcpb_orthogonalize_workspace_bytes(4, 4, None) == ARG
    assert lib.mhcpb_orthogonalize_workspace_bytes(4, TOO_WIDE, ctypes.byref(n)) == SHAPE
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    # one [T, F] of 16 bits, and for odd sizes the copies of x, the projections and w_down in padded rows
    assert m.mhc_ffn_forward_workspace_bytes(100, 64, 200) == up(100 * 200 * 2)
    assert m.mhc_ffn_forward_workspace_bytes(100, 65, 201) == up(100 * 208 * 2) + up(100 * 72 * 2) + 2 * up(201 * 72 * 2) + up(65 * 208 * 2)
    # up to 64 tokens also what its rounding lost, from row 64 on; of few tokens it is FP32, with no copies
    assert m.mhc_ffn_forward_workspace_bytes(40, 64, 200) == up((64 + 40) * 200 * 2)
    assert m.mhc_ffn_forward_workspace_bytes(2, 65, 201) == up(2 * 201 * 4)
    # dg, du and a; both inputs and all weights in padded rows
    assert m.mhc_ffn_backward_workspace_bytes(100, 64, 200) == 3 * up(100 * 200 * 2)
    assert m.mhc_ffn_backward_workspace_bytes(40, 64, 200) == up(40 * 200 * 2) + 2 * up((64 + 40) * 200 * 2)
    assert m.mhc_ffn_backward_workspace_bytes(100, 65, 201) == 3 * up(100 * 208 * 2) + 2 * up(100 * 72 * 2) + 2 * up(201 * 72 * 2) + up(65 * 208 * 2)
    # a short side of at most 32 is held on chip
    assert m.mhc_orthogonalize_workspace_bytes(24, 20480) == 0 == m.mhc_orthogonalize_workspace_bytes(5000, 32)
    assert m.mhc_orthogonalize_workspace_bytes(33, 40) > 33 * 40 * 8
    assert m.mhc_orthogonalize_workspace_bytes(5120, 12800) < 5120 * 12800 * 8 + 5120 * 5120 * 4 + (1 << 20)


def test_status_and_sites_in_a_normal_build(lib):
    checked, sites = abi.mhcpb_debug_checked_matrix_sites()
    assert checked is False and list(sites) == list(abi.MATRIX_FAMILIES) and set(sites.values()) == {0}
    assert lib.mhcpb_debug_checked_matrix_sites(None, None) == ARG
    assert lib.mhcpb_operators_device_status(None, 0) == ARG


def _t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


W = (_t(24, 16), _t(24, 16), _t(16, 24))
WS = _t(1 << 16, dtype=torch.uint8)


@pytest.mark.parametrize("call", [
    lambda: m.mhc_ffn_forward(_t(4, 16, dtype=F32), *(w.float() for w in W), _t(4, 16, dtype=F32), WS),
    lambda: m.mhc_ffn_forward(_t(4, 16, dtype=FP), *W, _t(4, 16, dtype=FP), WS),
    lambda: m.mhc_ffn_forward(_t(4, 17), *W, _t(4, 17), WS),
    lambda: m.mhc_ffn_forward(_t(4, 16), W[0], _t(23, 16), W[2], _t(4, 16), WS),
    lambda: m.mhc_ffn_forward(_t(4, 16), W[0], W[1], _t(24, 16), _t(4, 16), WS),
    lambda: m.mhc_ffn_forward(_t(4, 16), W[0], _t(16, 24).t(), W[2], _t(4, 16), WS),
    lambda: m.mhc_ffn_forward(_t(16, 4).t(), *W, _t(4, 16), WS),
    lambda: m.mhc_ffn_forward(_t(4, 16), *W, _t(5, 16), WS),
    lambda: m.mhc_ffn_forward(_t(4, 16), *W, _t(4, 16), WS, _t(4, 23), _t(4, 24)),
    lambda: m.mhc_ffn_forward(_t(4, 16), *W, _t(4, 16), WS, _t(4, 24, dtype=F32), _t(4, 24)),
    lambda: m.mhc_ffn_forward(_t(4, 16), *W, _t(4, 16), WS, activation="relu"),
    lambda: m.mhc_ffn_forward(_t(4, 16), *W, _t(4, 16), WS, activation=None),
    lambda: m.mhc_ffn_forward(_t(4, 16), *W, _t(4, 16), WS[::2]),
    lambda: m.mhc_ffn_forward(_t(64), *W, _t(4, 16), WS),
    lambda: m.mhc_ffn_backward(_t(4, 16), *W, _t(4, 24), _t(4, 24), _t(4, 16), _t(4, 16), _t(24, 16, dtype=FP), None, None, WS),
    lambda: m.mhc_ffn_backward(_t(4, 16), *W, _t(4, 24), _t(4, 24), _t(4, 16), None, _t(24, 16), _t(24, 16, dtype=F32), None, WS),
    lambda: m.mhc_ffn_backward(_t(4, 16), *W, _t(4, 24), _t(4, 24), _t(4, 16), None, None, None, _t(24, 16), WS),
    lambda: m.mhc_ffn_backward(_t(4, 16), *W, _t(4, 24), _t(3, 24), _t(4, 16), None, None, None, None, WS),
    lambda: m.mhc_orthogonalize(_t(4, 16), _t(4, 16, dtype=F32), WS),
    lambda: m.mhc_orthogonalize(_t(4, 16, dtype=torch.int32), _t(4, 16), WS),
    lambda: m.mhc_orthogonalize(_t(4, 16), _t(16, 4), WS),
    lambda: m.mhc_orthogonalize(_t(16, 4).t(), _t(4, 16), WS),
    lambda: m.mhc_orthogonalize(_t(64), _t(64), WS),
])
def test_python_checks(call):
    with pytest.raises(ValueError):
        call()


def test_one_pointer_of_gate_and_up_is_refused_in_python_too():
    with pytest.raises(abi.MhcpbError) as e:
        m.mhc_ffn_forward(_t(4, 16), *W, _t(4, 16), WS, _t(4, 24))
    assert e.value.status == ARG


def test_host_tensors_are_refused():
    with pytest.raises(abi.MhcpbError) as e:
        m.mhc_ffn_forward(_t(4, 16), *W, _t(4, 16), WS)
    assert e.value.status in (abi.MHCPB_ERR_WRONG_DEVICE, abi.MHCPB_ERR_CUDA)
