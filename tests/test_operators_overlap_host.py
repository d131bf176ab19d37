"""Overlapping operands of the operators around the stage, refused before any
CUDA call: the addresses below belong to nothing and are never read."""
import pytest

from rms_backward_gb300 import abi

A, B, C, FAR = 1 << 20, 2 << 20, 3 << 20, 64 << 20
T, D = 6, 8


def _status(call, *args):
    with pytest.raises(abi.MhcpbError) as e:   # without a GPU, or with these addresses, no call succeeds
        getattr(abi, call)(*args)
    return e.value.status


@pytest.mark.parametrize("call,args", [
    ("mhcpb_update_forward", (T, D, A, A, B, 0.0, None, 0, A, None)),        # y is the streams that are overwritten
    ("mhcpb_update_forward", (T, D, A, B, A, 0.0, None, 0, A, None)),        # h is
    ("mhcpb_update_forward", (T, D, A, B, C, 0.5, A, 0, A, None)),           # the generator's state is
    ("mhcpb_dropout", (64, abi.MHCPB_BF16, A, 0.5, A, 0, A, None)),
])
def test_in_place_excuses_one_operand_only(call, args):
    """x_out may be x, and dropout's y its x; another operand at that address is
    overwritten while it is read."""
    assert _status(call, *args) == abi.MHCPB_ERR_ALIASING


@pytest.mark.parametrize("call,args", [
    ("mhcpb_update_forward", (T, D, A, B, C, 0.5, FAR, 0, A, None)),
    ("mhcpb_update_forward", (T, D, A, A, C, 0.0, None, 0, B, None)),        # inputs may share memory
    ("mhcpb_dropout", (64, abi.MHCPB_BF16, A, 0.5, FAR, 0, A, None)),
])
def test_in_place_is_not_an_overlap(call, args):
    assert _status(call, *args) != abi.MHCPB_ERR_ALIASING


def _norm_status(x, x_stride, y, y_stride, width=D, type_=abi.MHCPB_BF16):
    return _status("mhcpb_layernorm_forward", T, width, type_, x, x_stride, None, None, 1e-5, y, y_stride, None, None, None)


def _gradient_status(x, gy, gx, stride, width=D):
    return _status("mhcpb_layernorm_backward", T, width, abi.MHCPB_FP32, x, stride, gy, stride, None, B, C, gx, stride,
                   None, None, 0, None, 0, None)


# (byte offset of y from x, row strides in elements of 2 bytes): 8 columns, 16 bytes a row
@pytest.mark.parametrize("offset,x_stride,y_stride", [
    (16, 16, 16), (-16, 16, 16), (16, 17, 17), (18, 17, 17),       # column slices of one buffer, either first
    (16 + 3 * 48, 24, 24), (-32 - 2 * 48, 24, 24),                 # and some rows further on
    (-16 - 5 * 32, 16, 16), (6 * 32, 16, 16), (6 * 16, 8, 8),      # one after the other
])
def test_rows_between_rows_do_not_overlap(offset, x_stride, y_stride):
    assert _norm_status(A, x_stride, A + offset, y_stride) != abi.MHCPB_ERR_ALIASING


@pytest.mark.parametrize("offset,x_stride,y_stride", [
    (0, 16, 16), (14, 16, 16), (-14, 16, 16), (32, 16, 16), (14 + 3 * 32, 16, 16), (-2 - 2 * 32, 16, 16),
    (2, 8, 8), (20, 17, 17), (16 + 34, 17, 16), (16, 16, 17), (16, 32, 16),
])
def test_rows_that_share_columns_overlap(offset, x_stride, y_stride):
    assert _norm_status(A, x_stride, A + offset, y_stride) == abi.MHCPB_ERR_ALIASING


def test_gradients_in_slices_of_one_buffer():
    assert _gradient_status(A, A + 32, A + 64, 24) != abi.MHCPB_ERR_ALIASING
    assert _gradient_status(A, A, A + 64, 24) != abi.MHCPB_ERR_ALIASING        # inputs may share memory
    assert _gradient_status(A, A + 32, A + 60, 24) == abi.MHCPB_ERR_ALIASING
    assert _gradient_status(A, A + 64, A + 32 + 24 * 4 * 4, 24) != abi.MHCPB_ERR_ALIASING
