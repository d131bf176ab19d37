"""Host-side refusals of the operators around the stage: bad shapes, types,
flags and probabilities before any CUDA call, and the Python layer's checks of
types, shapes and strides (all without a GPU)."""
import ctypes
import os

import pytest
import torch

import rms_backward_gb300 as m
from rms_backward_gb300 import abi

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from rms_backward_gb300 import build
        build.build()
    return abi.load()


SHAPE, ARG = abi.MHCPB_ERR_UNSUPPORTED_SHAPE, abi.MHCPB_ERR_INVALID_ARG
TOO_LONG, TOO_WIDE = (1 << 24) + 1, (1 << 20) + 1


@pytest.mark.parametrize("status,call,args", [
    (SHAPE, "mhcpb_embed_forward", (-1, 5, 8, 4, 0, 0, 0, 8, 1.0, 0, None)),
    (SHAPE, "mhcpb_embed_forward", (1, 0, 8, 4, 0, 0, 0, 8, 1.0, 0, None)),
    (SHAPE, "mhcpb_embed_forward", (1, TOO_LONG, 8, 4, 0, 0, 0, 8, 1.0, 0, None)),
    (SHAPE, "mhcpb_embed_forward", (1, 5, 8, 17, 0, 0, 0, 8, 1.0, 0, None)),
    (SHAPE, "mhcpb_embed_forward", (1, 5, (1 << 18) + 1, 4, 0, 0, 0, 8, 1.0, 0, None)),
    (ARG, "mhcpb_embed_forward", (1, 5, 8, 4, 3, 0, 0, 8, 1.0, 0, None)),
    (ARG, "mhcpb_embed_forward", (1, 5, 8, 4, 0, 0, 0, 2, 1.0, 0, None)),
    (ARG, "mhcpb_embed_forward", (1, 5, 8, 4, 0, 0, 0, 8, 1.0, 0, None)),   # NULL operands
    (ARG, "mhcpb_embed_backward", (1, 5, 8, 4, 0, 0, 8, 1.0, 1, 0, 0, 1 << 30, None)),
    (SHAPE, "mhcpb_embed_backward", (1, 5, 0, 4, 0, 0, 8, 1.0, 0, 0, 0, 1 << 30, None)),
    (abi.MHCPB_ERR_WORKSPACE_TOO_SMALL, "mhcpb_embed_backward", (1, 5, 8, 4, 0, 0, 8, 1.0, 0, 0, 0, 0, None)),
    (SHAPE, "mhcpb_embed_workspace_bytes", (1, 5, TOO_WIDE)),
    (SHAPE, "mhcpb_layernorm_forward", (TOO_LONG, 8, 0, 0, 8, 0, 0, 1e-5, 0, 8, 0, 0, None)),
    (SHAPE, "mhcpb_layernorm_forward", (1, TOO_WIDE, 0, 0, TOO_WIDE, 0, 0, 1e-5, 0, TOO_WIDE, 0, 0, None)),
    (SHAPE, "mhcpb_layernorm_forward", (1, 8, 0, 0, 7, 0, 0, 1e-5, 0, 8, 0, 0, None)),
    (SHAPE, "mhcpb_layernorm_forward", (1, 8, 0, 0, 8, 0, 0, 1e-5, 0, TOO_LONG, 0, 0, None)),
    (ARG, "mhcpb_layernorm_forward", (1, 8, 0, 0, 8, 0, 0, -1.0, 0, 8, 0, 0, None)),
    (ARG, "mhcpb_layernorm_forward", (1, 8, 0, 0, 8, 0, 0, float("nan"), 0, 8, 0, 0, None)),
    (ARG, "mhcpb_layernorm_forward", (1, 8, -1, 0, 8, 0, 0, 1e-5, 0, 8, 0, 0, None)),
    (ARG, "mhcpb_layernorm_backward", (1, 8, 0, 0, 8, 0, 8, 0, 0, 0, 0, 8, 0, 0, 1 << 20, 0, 0, None)),
    (SHAPE, "mhcpb_layernorm_backward", (1, 8, 0, 0, 8, 0, -8, 0, 0, 0, 0, 8, 0, 0, 0, 0, 0, None)),
    (SHAPE, "mhcpb_layernorm_workspace_bytes", (-1, 8)),
    (ARG, "mhcpb_dropout", (8, 0, 0, 1.0, 0, 0, 0, None)),
    (ARG, "mhcpb_dropout", (8, 0, 0, -0.1, 0, 0, 0, None)),
    (ARG, "mhcpb_dropout", (8, 0, 0, float("nan"), 0, 0, 0, None)),
    (ARG, "mhcpb_dropout", (8, 9, 0, 0.1, 0, 0, 0, None)),
    (SHAPE, "mhcpb_dropout", (-8, 0, 0, 0.1, 0, 0, 0, None)),
    (SHAPE, "mhcpb_collapse_norm_forward", (1, (1 << 18) + 1, 0, 0, 0, 0, 1e-5, 0, 0, 0, None)),
    (ARG, "mhcpb_collapse_norm_forward", (1, 8, 0, 0, 0, 0, float("inf"), 0, 0, 0, None)),
    (ARG, "mhcpb_collapse_norm_backward", (1, 8, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 8, 0, 0, None)),
    (SHAPE, "mhcpb_collapse_norm_workspace_bytes", (1, 0)),
    (SHAPE, "mhcpb_update_forward", (1, 0, 0, 0, 0, 0.0, 0, 0, 0, None)),
    (ARG, "mhcpb_update_forward", (1, 8, 0, 0, 0, 1.5, 0, 0, 0, None)),
    (SHAPE, "mhcpb_update_backward", (-2, 8, 0, 0, 0, 0.0, 0, 0, 0, 0, 0, None)),
])
def test_refused_before_cuda(status, call, args):
    with pytest.raises(abi.MhcpbError) as e:
        getattr(abi, call)(*args)
    assert e.value.status == status


def test_workspace_sizes(lib):
    n = ctypes.c_size_t()
    for f, k in (("embed", 3), ("layernorm", 2), ("collapse_norm", 2)):
        fn = getattr(lib, f"mhcpb_{f}_workspace_bytes")
        assert fn(*[4] * k, None) == ARG
        assert fn(0, *[4] * (k - 1), ctypes.byref(n)) == abi.MHCPB_OK and n.value == 0
        assert fn(*[4] * k, ctypes.byref(n)) == abi.MHCPB_OK and n.value > 0
    # order (two buffers) and a list of chunks, in 256-byte multiples, and two FP32 rows (of whole vectors) per chunk of ordered tokens
    assert m.mhc_embed_workspace_bytes(33, 7, 10) == 2 * 512 + 256 + 9 * 2 * 16 * 4
    assert m.mhc_embed_workspace_bytes(4096, 7, 10) == 2 * 32768 + 1280 + 256 * 2 * 16 * 4


def test_checked_operator_sites_in_a_normal_build(lib):
    checked, sites = abi.mhcpb_debug_checked_operator_sites()
    assert checked is False and list(sites) == list(abi.OPERATOR_FAMILIES) and set(sites.values()) == {0}
    assert lib.mhcpb_debug_checked_operator_sites(None, None) == ARG


def _t(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("call", [
    lambda: m.mhc_embed_forward(_t(3, dtype=torch.int16), _t(5, 8), _t(3, 8)),
    lambda: m.mhc_embed_forward(_t(6, dtype=torch.int64)[::2], _t(5, 8), _t(3, 8)),
    lambda: m.mhc_embed_forward(_t(3, dtype=torch.int64), _t(5, 8), _t(3, 12)),
    lambda: m.mhc_embed_forward(_t(3, dtype=torch.int64), _t(5, 8), _t(4, 8)),
    lambda: m.mhc_embed_forward(_t(3, dtype=torch.int64), _t(8, 5).t(), _t(3, 8)),
    lambda: m.mhc_embed_forward(_t(3, dtype=torch.int64), _t(5, 8, dtype=torch.float64), _t(3, 8)),
    lambda: m.mhc_embed_backward(_t(3, dtype=torch.int64), _t(3, 8), _t(5, 8), _t(9, dtype=torch.uint8)),
    lambda: m.mhc_layernorm_forward(_t(3, 8), None, None, _t(3, 8, dtype=torch.float32)),
    lambda: m.mhc_layernorm_forward(_t(8, 3).t(), None, None, _t(3, 8)),
    lambda: m.mhc_layernorm_forward(_t(3, 8), _t(8), None, _t(3, 8)),
    lambda: m.mhc_layernorm_forward(_t(3, 8), None, None, _t(3, 8), _t(4, dtype=torch.float32), None),
    lambda: m.mhc_layernorm_backward(_t(3, 8), _t(3, 7), None, *[_t(3, dtype=torch.float32)] * 2, _t(3, 8)),
    lambda: m.mhc_dropout(_t(8), _t(9), p=0.0),
    lambda: m.mhc_dropout(_t(8, dtype=torch.int32), _t(8), p=0.0),
    lambda: m.mhc_dropout(_t(8), _t(8), p=0.5),
    lambda: m.mhc_dropout(_t(8), _t(8), _t(3, dtype=torch.int64), p=0.5),
    lambda: m.mhc_collapse_norm_forward(_t(3, 30), _t(3, 24, dtype=torch.float32), None, None, _t(3, 8)),
    lambda: m.mhc_collapse_norm_forward(_t(3, 32), _t(2, 24, dtype=torch.float32), None, None, _t(3, 8)),
    lambda: m.mhc_update_forward(_t(3, 32), _t(3, 32), _t(3, 24, dtype=torch.float32), _t(3, 32)),
    lambda: m.mhc_update_backward(_t(3, 32), _t(3, 8), _t(3, 24), _t(3, 32), _t(3, 8), _t(3, 24)),
])
def test_python_checks(call):
    with pytest.raises(ValueError):
        call()


def test_workspaces_are_compact():
    """A workspace's size is its bytes, so it has to hold them: none that is expanded or strided."""
    f32 = lambda *s: _t(*s, dtype=torch.float32)  # noqa: E731
    for ws in (_t(1, dtype=torch.uint8).expand(1 << 20), _t(1 << 20, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="workspace"):
            m.mhc_embed_backward(_t(3, dtype=torch.int64), _t(3, 8), f32(5, 8), ws)
        with pytest.raises(ValueError, match="workspace"):
            m.mhc_layernorm_backward(_t(3, 8), _t(3, 8), f32(8), f32(3), f32(3), _t(3, 8), f32(8), f32(8), ws)
        with pytest.raises(ValueError, match="workspace"):
            m.mhc_collapse_norm_backward(_t(3, 32), f32(3, 24), _t(3, 8), f32(8), f32(3), f32(3), _t(3, 32), f32(3, 24),
                                         f32(8), f32(8), ws)
