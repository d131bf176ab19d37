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
