"""Binding of the operators around a training step (include/dpr_step.h): the
RMS norm with the residual's addition, the linear layers of experts, and the
norm and clipping of gradients.  Tensors, checks and scratch memory are those
of the backward-pass operators (_operators.py).
"""
from __future__ import annotations

import ctypes
from typing import Sequence

import torch

from ._binding import _check, _ptrs, _stream, lib
from ._operators import (_DTYPES, _checkpoint_arg, _code, _device, _handle, _matrix, _statistic,
                         _vector, _workspace, _workspace_bytes, _wrong_device, _wrong_shape)


def _experts(t: torch.Tensor, what: str, dev: int):
    """(address, experts, rows, width, row stride, expert stride) of [experts, rows, width]."""
    if t.get_device() != dev:
        _wrong_device(t, what)
    if t.dim() != 3 or t.shape[0] == 0:
        raise ValueError(f"{what}: need [experts, out_features, in_features], got {tuple(t.shape)}")
    experts, rows, width = t.shape
    outer, stride, inner = t.stride()
    if inner != 1 and width > 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    stride = stride if rows > 1 or stride > width else width
    return (t.data_ptr(), experts, rows, width, stride,
            outer if experts > 1 else rows * stride)


def _bf16(t: torch.Tensor, what: str):
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{what}: need torch.bfloat16, got {t.dtype}")


def _offsets(t: torch.Tensor, experts: int, dev: int) -> int:
    """Address of the experts' offsets."""
    if t.dtype != torch.int32:
        raise ValueError(f"offsets: need torch.int32, got {t.dtype}")
    return _vector(t, experts + 1, "offsets", dev)


def _grouped_product(fn: str, x, what: str, offsets, weight, out, out_what: str, workspace, stream):
    """The product and its input gradient, which differ in the side of the
    weight that their argument and their result have."""
    dev = _device(x, what)
    px, rows, width, sx = _matrix(x, what, dev)
    _bf16(x, what)
    _bf16(weight, "weight")
    pw, experts, o, i, sw, ew = _experts(weight, "weight", dev)
    have, give = (i, o) if fn == "dpr_grouped_linear" else (o, i)
    if width != have:
        raise ValueError(f"{what}: rows of {width}, but weight is {tuple(weight.shape)}")
    po, r, w, so = _matrix(out, out_what, dev)
    if r != rows or w != give:
        _wrong_shape(out_what, r, w, rows, give)
    offs = _offsets(offsets, experts, dev)
    need = ctypes.c_int64()
    L = lib()
    st = getattr(L, fn + "_workspace")(px, sx, rows, experts, pw, sw, ew, o, i, ctypes.byref(need))
    if st:
        _check(fn, st)
    nbytes = need.value
    handle = _handle(stream, dev)
    ws = _workspace(workspace, nbytes, stream, handle, dev)
    st = getattr(L, fn)(px, sx, rows, offs, experts, pw, sw, ew, o, i, po, so, _code(out, out_what),
                        0 if ws is None else ws.data_ptr(), nbytes, handle)
    if st:
        _check(fn, st)


def dpr_grouped_linear(x: torch.Tensor, offsets: torch.Tensor, weight: torch.Tensor,
                       y: torch.Tensor, workspace=None, stream=None) -> None:
    """y[t] = weight[e] x[t] for the rows offsets[e] .. offsets[e + 1] - 1 of
    each expert e: x bf16 [..., in_features], offsets int32 [experts + 1] on
    the device, weight bf16 [experts, out_features, in_features], y bf16 or
    fp32.  Rows of y that belong to no expert are left as they are."""
    _grouped_product("dpr_grouped_linear", x, "x", offsets, weight, y, "y", workspace, stream)


def dpr_grouped_linear_input_grad(dy: torch.Tensor, offsets: torch.Tensor, weight: torch.Tensor,
                                  dx: torch.Tensor, workspace=None, stream=None) -> None:
    """dx[t] = weight[e]^T dy[t], the input gradient of dpr_grouped_linear."""
    _grouped_product("dpr_grouped_linear_input_grad", dy, "dy", offsets, weight, dx, "dx",
                     workspace, stream)


def dpr_grouped_linear_weight_grad(dy: torch.Tensor, offsets: torch.Tensor, x,
                                   dweight: torch.Tensor, accumulate: bool = False,
                                   workspace=None, stream=None) -> None:
    """dweight[e] = sum over expert e's tokens of dy[t] x[t]^T, with dy bf16
    [..., out_features] and x bf16 [..., in_features] or its Checkpoint;
    dweight bf16 or fp32 [experts, out_features, in_features], added to with
    `accumulate`.  Experts without tokens get zeros."""
    dev = _device(dy, "dy")
    pd, rows, out_features, sd = _matrix(dy, "dy", dev)
    _bf16(dy, "dy")
    pw, experts, o, in_features, sw, ew = _experts(dweight, "dweight", dev)
    if o != out_features:
        raise ValueError(f"dweight: {o} rows, but dy has {out_features} out-features")
    px = sx = 0
    ref = None
    if isinstance(x, torch.Tensor):
        px, r, w, sx = _matrix(x, "x", dev)
        _bf16(x, "x")
        if r != rows or w != in_features:
            _wrong_shape("x", r, w, rows, in_features)
    else:
        ref = ctypes.byref(_checkpoint_arg(x, "x", rows, in_features, dev))
    offs = _offsets(offsets, experts, dev)
    need = ctypes.c_int64()
    L = lib()
    st = L.dpr_grouped_linear_weight_grad_workspace(pd, sd, px, sx, ref, rows, experts, out_features,
                                                    in_features, ctypes.byref(need))
    if st:
        _check("dpr_grouped_linear_weight_grad", st)
    nbytes = need.value
    handle = _handle(stream, dev)
    ws = _workspace(workspace, nbytes, stream, handle, dev)
    st = L.dpr_grouped_linear_weight_grad(
        pd, sd, px, sx, ref, rows, offs, experts, out_features, in_features, pw, sw, ew,
        _code(dweight, "dweight"), 1 if accumulate else 0, 0 if ws is None else ws.data_ptr(),
        nbytes, handle)
    if st:
        _check("dpr_grouped_linear_weight_grad", st)
