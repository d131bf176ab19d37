"""The texts that an error shows to a user hold for every call that returns
its status: a plan's calls and the operators around the stage, which have no
plan, take any hidden size and no token, and want less alignment."""
import pytest

from rms_backward_gb300 import abi


def _message(call, *args):
    with pytest.raises(abi.MhcpbError) as e:
        getattr(abi, call)(*args)
    return e.value.status, str(e.value)


@pytest.mark.parametrize("status,call,args", [
    # ids one byte off, of 8
    (abi.MHCPB_ERR_MISALIGNED, "mhcpb_embed_forward", (2, 2, 8, 4, 0, 4096, 8193, 8, 1.0, 16384, None)),
    # a row stride below the row; too many streams; a table too long
    (abi.MHCPB_ERR_UNSUPPORTED_SHAPE, "mhcpb_layernorm_forward", (1, 8, 0, 0, 7, 0, 0, 1e-5, 0, 8, 0, 0, None)),
    (abi.MHCPB_ERR_UNSUPPORTED_SHAPE, "mhcpb_embed_forward", (1, 5, 8, 17, 0, 0, 0, 8, 1.0, 0, None)),
    (abi.MHCPB_ERR_UNSUPPORTED_SHAPE, "mhcpb_embed_workspace_bytes", (1, (1 << 24) + 1, 8)),
])
def test_operator_errors_state_no_rule_of_the_plan(status, call, args):
    got, text = _message(call, *args)
    assert got == status
    for wrong in ("16-byte", "T >= 1", "multiple of 8", "plan"):
        assert wrong not in text, text


def test_wrong_device_text_needs_no_plan():
    assert "plan" not in abi.status_string(abi.MHCPB_ERR_WRONG_DEVICE)
