"""The operators around the projection stage on torch CUDA tensors: embedding
into the residual streams, layer norm, dropout, stream collapse with its norm,
and stream update, each with its gradient (``include/mhcpb.h`` has the
formulas).

Every function writes into tensors the caller passes and returns nothing; it
allocates nothing and does not wait.  Types, shapes and strides are checked
here (``ValueError``); pointers, alignment, overlap and device in the library
(``MhcpbError``).  ``stream`` is a ``torch.cuda.Stream``, a raw handle, or None
for the current stream; tensors made on another stream are ordered by the
caller, as for any torch kernel.  BF16 streams x are [T, 4 D] with stream s in
columns s D .. (s + 1) D - 1, gates h are FP32 [T, 24] as the gate step writes
them, parameters and their gradients are FP32.
"""
from __future__ import annotations

import torch

from . import abi

N_STREAMS = 4
_TYPES = {torch.bfloat16: abi.MHCPB_BF16, torch.float16: abi.MHCPB_FP16, torch.float32: abi.MHCPB_FP32}
_BF16, _F32 = torch.bfloat16, torch.float32


_raw_stream = torch._C._cuda_getCurrentRawStream


def _handle(stream, like):
    if stream is None:
        device = like.get_device()
        return _raw_stream(device) if device >= 0 else None   # the library refuses host tensors
    return getattr(stream, "cuda_stream", stream)


def _lib():
    return abi._lib or abi.load()


def _need(t, name, shape, dtype):
    """t is a compact tensor of this shape and type."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()}")
    return t.data_ptr()


def _compact(t, name, dtype=None):
    """t is a compact tensor (of this type, where given)."""
    if (dtype is not None and t.dtype is not dtype) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype or t.dtype} tensor, got {t.dtype} {tuple(t.shape)} "
                         f"with strides {t.stride()}")
    return t.data_ptr()


def _scratch(workspace):
    """(pointer, bytes) of a workspace, or of none."""
    if workspace is None:
        return None, 0
    return _compact(workspace, "workspace"), workspace.nbytes


def _maybe(t, name, shape, dtype):
    return None if t is None else _need(t, name, shape, dtype)


def _rows(t, name, shape, dtype):
    """(pointer, row stride) of a [T, D] tensor whose rows are compact."""
    if t.dtype is dtype and t.is_contiguous() and t.shape == shape:
        return t.data_ptr(), shape[1]
    if t.dtype is not dtype or t.shape != shape or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected a {dtype} tensor of shape {tuple(shape)} with compact rows, "
                         f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()}")
    return t.data_ptr(), (t.stride(0) if shape[0] > 1 else shape[1])


def _type(t, name):
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{name}: expected bfloat16, float16 or float32, got {t.dtype}") from None


def _two_dims(t, name):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: expected a [T, D] tensor, got shape {tuple(shape)}")
    return shape


def _streams(x, name):
    T, K = _two_dims(x, name)
    if K % N_STREAMS or K == 0:
        raise ValueError(f"{name}: expected [T, {N_STREAMS} D] streams, got shape {tuple(x.shape)}")
    return T, K // N_STREAMS


def _rng(rng, p):
    if p == 0:
        return None
    if rng is None:
        raise ValueError("rng: dropout with p > 0 needs the generator state, an int64 tensor {key, step}")
    return _need(rng, "rng", (2,), torch.int64)


def _ids(ids, table_shape, x, name):
    if ids.dtype not in (torch.int32, torch.int64) or ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError(f"ids: expected a contiguous [T] int32 or int64 tensor, got {ids.dtype} {tuple(ids.shape)}")
    T, K = _two_dims(x, name)
    D = table_shape[1]
    if D == 0 or K % D or T != ids.shape[0]:
        raise ValueError(f"{name}: expected [{ids.shape[0]}, n_streams * {D}], got {tuple(x.shape)}")
    return T, D, K // D


# ---------------------------------------------------------------- embedding
def mhc_embed_forward(ids, table, x, *, scale: float = 1.0, stream=None):
    """x[t, s, :] = bf16(scale * table[ids[t], :]) for every stream s: ids [T]
    int32 or int64, table [V, D] BF16, FP16 or FP32, x BF16 [T, n_streams D].
    Ids outside [0, V) give rows of zeros."""
    V, _ = _two_dims(table, "table")
    T, D, n = _ids(ids, table.shape, x, "x")
    status = _lib().mhcpb_embed_forward(T, V, D, n, _type(table, "table"), _compact(table, "table"),
                                        ids.data_ptr(), ids.element_size(), scale, _compact(x, "x", _BF16),
                                        _handle(stream, x))
    if status:
        abi._check(status, "mhcpb_embed_forward")


def mhc_embed_workspace_bytes(T: int, V: int, D: int) -> int:
    """Scratch bytes of :func:`mhc_embed_backward`."""
    return abi.mhcpb_embed_workspace_bytes(T, V, D)


def mhc_embed_backward(ids, grad_x, grad_table, workspace, *, scale: float = 1.0, accumulate: bool = False,
                       stream=None):
    """grad_table [V, D] FP32 = scale * the sum of grad_x [T, n_streams D] BF16
    over the tokens of each row and the streams (added to it with
    ``accumulate``), summed in a fixed order."""
    V, _ = _two_dims(grad_table, "grad_table")
    T, D, n = _ids(ids, grad_table.shape, grad_x, "grad_x")
    status = _lib().mhcpb_embed_backward(T, V, D, n, _compact(grad_x, "grad_x", _BF16), ids.data_ptr(),
                                         ids.element_size(), scale, abi.MHCPB_ACCUMULATE_DW if accumulate else 0,
                                         _compact(grad_table, "grad_table", _F32), *_scratch(workspace),
                                         _handle(stream, grad_x))
    if status:
        abi._check(status, "mhcpb_embed_backward")


# ---------------------------------------------------------------- layer norm
def mhc_layernorm_forward(x, gamma, beta, y, mean=None, rstd=None, *, eps: float = 1e-5, stream=None):
    """y = (x - mean) * rstd * gamma + beta over the last axis of x [T, D] (BF16,
    FP16 or FP32; x and y may have a row stride).  gamma, beta: FP32 [D] or
    None; mean, rstd: FP32 [T], both None where no backward follows."""
    T, D = shape = _two_dims(x, "x")
    dtype = x.dtype
    xp, xs = _rows(x, "x", shape, dtype)
    yp, ys = _rows(y, "y", shape, dtype)
    status = _lib().mhcpb_layernorm_forward(T, D, _type(x, "x"), xp, xs, _maybe(gamma, "gamma", (D,), _F32),
                                            _maybe(beta, "beta", (D,), _F32), eps, yp, ys,
                                            _maybe(mean, "mean", (T,), _F32), _maybe(rstd, "rstd", (T,), _F32),
                                            _handle(stream, x))
    if status:
        abi._check(status, "mhcpb_layernorm_forward")


def mhc_layernorm_workspace_bytes(T: int, D: int) -> int:
    """Scratch bytes of :func:`mhc_layernorm_backward` with parameter gradients."""
    return abi.mhcpb_layernorm_workspace_bytes(T, D)


def mhc_layernorm_backward(x, grad_y, gamma, mean, rstd, grad_x, grad_gamma=None, grad_beta=None, workspace=None, *,
                           accumulate: bool = False, stream=None):
    """grad_x, and grad_gamma and grad_beta where given (added to with
    ``accumulate``), from the forward's x, mean and rstd."""
    T, D = shape = _two_dims(x, "x")
    dtype = x.dtype
    xp, xs = _rows(x, "x", shape, dtype)
    gp, gs = _rows(grad_y, "grad_y", shape, dtype)
    dp, ds = _rows(grad_x, "grad_x", shape, dtype)
    status = _lib().mhcpb_layernorm_backward(T, D, _type(x, "x"), xp, xs, gp, gs, _maybe(gamma, "gamma", (D,), _F32),
                                             _need(mean, "mean", (T,), _F32), _need(rstd, "rstd", (T,), _F32), dp, ds,
                                             _maybe(grad_gamma, "grad_gamma", (D,), _F32),
                                             _maybe(grad_beta, "grad_beta", (D,), _F32),
                                             abi.MHCPB_ACCUMULATE_DW if accumulate else 0,
                                             *_scratch(workspace), _handle(stream, x))
    if status:
        abi._check(status, "mhcpb_layernorm_backward")


# ---------------------------------------------------------------- dropout
def mhc_dropout(x, y, rng=None, *, p: float, sequence: int = 0, stream=None):
    """y = x / (1 - p) where kept, else 0; the mask comes from ``rng`` (an int64
    CUDA tensor {key, step}), ``sequence`` and the element's index, so the same
    call on the gradient is the gradient.  y may be x."""
    status = _lib().mhcpb_dropout(x.numel(), _type(x, "x"), _compact(x, "x"), p, _rng(rng, p), sequence,
                                  _need(y, "y", x.shape, x.dtype), _handle(stream, x))
    if status:
        abi._check(status, "mhcpb_dropout")


# ---------------------------------------------------------------- collapse and norm
def mhc_collapse_norm_forward(x, h, gamma, beta, y, mean=None, rstd=None, *, eps: float = 1e-5, stream=None):
    """y = layer norm of sum_s h[:, s] x_s: the sublayer's input [T, D] BF16."""
    T, D = _streams(x, "x")
    status = _lib().mhcpb_collapse_norm_forward(T, D, _compact(x, "x", _BF16), _need(h, "h", (T, 24), _F32),
                                                _maybe(gamma, "gamma", (D,), _F32),
                                                _maybe(beta, "beta", (D,), _F32), eps,
                                                _need(y, "y", (T, D), _BF16), _maybe(mean, "mean", (T,), _F32),
                                                _maybe(rstd, "rstd", (T,), _F32), _handle(stream, x))
    if status:
        abi._check(status, "mhcpb_collapse_norm_forward")


def mhc_collapse_norm_workspace_bytes(T: int, D: int) -> int:
    """Scratch bytes of :func:`mhc_collapse_norm_backward` with parameter gradients."""
    return abi.mhcpb_collapse_norm_workspace_bytes(T, D)


def mhc_collapse_norm_backward(x, h, grad_y, gamma, mean, rstd, grad_x, grad_h, grad_gamma=None, grad_beta=None,
                               workspace=None, *, grad_x_out=None, accumulate: bool = False, stream=None):
    """grad_x [T, 4 D] (with the residual path's share H_res^T grad_x_out, where
    given) and columns 0..3 of grad_h [T, 24] from grad_y [T, D]."""
    T, D = _streams(x, "x")
    status = _lib().mhcpb_collapse_norm_backward(
        T, D, _compact(x, "x", _BF16), _need(h, "h", (T, 24), _F32), _need(grad_y, "grad_y", (T, D), _BF16),
        _maybe(gamma, "gamma", (D,), _F32), _need(mean, "mean", (T,), _F32), _need(rstd, "rstd", (T,), _F32),
        _maybe(grad_x_out, "grad_x_out", x.shape, _BF16), _need(grad_x, "grad_x", x.shape, _BF16),
        _need(grad_h, "grad_h", (T, 24), _F32), _maybe(grad_gamma, "grad_gamma", (D,), _F32),
        _maybe(grad_beta, "grad_beta", (D,), _F32), abi.MHCPB_ACCUMULATE_DW if accumulate else 0,
        *_scratch(workspace), _handle(stream, x))
    if status:
        abi._check(status, "mhcpb_collapse_norm_backward")


# ---------------------------------------------------------------- stream update
def mhc_update_forward(x, y, h, x_out, rng=None, *, p: float = 0.0, sequence: int = 0, stream=None):
    """x_out_i = sum_j H_res[i, j] x_j + H_post[i] dropout(y), H_post and H_res
    from h [T, 24]; x_out may be x."""
    T, D = _streams(x, "x")
    status = _lib().mhcpb_update_forward(T, D, _compact(x, "x", _BF16), _need(y, "y", (T, D), _BF16),
                                         _need(h, "h", (T, 24), _F32), p, _rng(rng, p), sequence,
                                         _need(x_out, "x_out", x.shape, _BF16), _handle(stream, x))
    if status:
        abi._check(status, "mhcpb_update_forward")


def mhc_update_backward(x, y, h, grad_x_out, grad_y, grad_h, rng=None, *, p: float = 0.0, sequence: int = 0,
                        stream=None):
    """grad_y [T, D] and columns 4..23 of grad_h [T, 24] from grad_x_out [T, 4 D];
    the streams' own gradient is :func:`mhc_collapse_norm_backward`'s."""
    T, D = _streams(x, "x")
    status = _lib().mhcpb_update_backward(T, D, _compact(x, "x", _BF16), _need(y, "y", (T, D), _BF16),
                                          _need(h, "h", (T, 24), _F32), p, _rng(rng, p), sequence,
                                          _need(grad_x_out, "grad_x_out", x.shape, _BF16),
                                          _need(grad_y, "grad_y", (T, D), _BF16),
                                          _need(grad_h, "grad_h", (T, 24), _F32), _handle(stream, x))
    if status:
        abi._check(status, "mhcpb_update_backward")
