"""Binding of the operators around a training step (include/dpr_step.h): the
RMS norm with the residual's addition, the linear layers of experts, and the
norm and clipping of gradients.  Tensors, checks and scratch memory are those
of the backward-pass operators (_operators.py).
"""
from __future__ import annotations

import ctypes
import functools
from typing import Sequence

import torch

from ._binding import _check, _ptrs, _stream, lib
from ._operators import (_DTYPES, _CheckpointArg, _checkpoint_arg, _code, _device, _handle, _matrix, _statistic,
                         _vector, _workspace, _workspace_bytes, _wrong_device, _wrong_shape)


def _like(t, shape, rows: int, width: int, dtype, what: str, dev: int):
    """(address, row stride) of a matrix of `rows` x `width` and this type;
    zeros for None.  A tensor of the call's own shape takes the short way."""
    if t is None:
        return 0, 0
    if t.dtype != dtype:
        raise ValueError(f"{what}: need {dtype}, got {t.dtype}")
    if len(shape) == 2 and t.shape == shape and t.get_device() == dev:
        stride, inner = t.stride()
        if inner == 1 and stride >= width:
            return t.data_ptr(), stride
    p, r, w, stride = _matrix(t, what, dev)
    if r != rows or w != width:
        _wrong_shape(what, r, w, rows, width)
    return p, stride


def _saved(c, what: str, rows: int, width: int, dev: int):
    return None if c is None else ctypes.byref(_checkpoint_arg(c, what, rows, width, dev))


def dpr_rmsnorm_forward(x: torch.Tensor, weight, eps: float, y=None, rstd=None, residual=None,
                        h=None, h_checkpoint=None, y_checkpoint=None, stream=None) -> None:
    """h = x + residual (rounded to their type; x without a residual) and y = h *
    rstd * weight, rstd = 1 / sqrt(mean(h^2) + eps), along the last dimension;
    weight (bf16 or fp32) may be None.  h, where the residual stream goes on,
    may be x or residual; y may be x or residual too.  rstd ([rows] fp32) is
    what the backward pass needs.  The checkpoints are written in the same pass
    as dpr_checkpoint_save(h) and (y) would; with y_checkpoint y may be None."""
    dev = _device(x, "x")
    px, rows, width, sx = _matrix(x, "x", dev)
    shape, dtype = x.shape, x.dtype
    pr, sr = _like(residual, shape, rows, width, dtype, "residual", dev)
    ph, sh = _like(h, shape, rows, width, dtype, "h", dev)
    py, sy = _like(y, shape, rows, width, dtype, "y", dev)
    st = lib().dpr_rmsnorm_forward(
        px, sx, pr, sr, rows, width, _code(x, "x"), _vector(weight, width, "weight", dev),
        0 if weight is None else _code(weight, "weight"), eps, ph, sh, py, sy,
        _statistic(rstd, rows, "rstd", dev), _saved(h_checkpoint, "h_checkpoint", rows, width, dev),
        _saved(y_checkpoint, "y_checkpoint", rows, width, dev), _handle(stream, dev))
    if st:
        _check("dpr_rmsnorm_forward", st)


def dpr_rmsnorm_backward(dy: torch.Tensor, h, weight, rstd: torch.Tensor, dx: torch.Tensor,
                         dweight=None, dh=None, accumulate: bool = False, workspace=None,
                         stream=None) -> None:
    """dx and dweight of dpr_rmsnorm_forward.  `h` is the forward's sum (its x
    without a residual) or its Checkpoint; `dh` the gradient that reaches h
    past the norm, added to dx.  dx, the gradient of x and of the residual, may
    be dy, dh or h.  dweight (bf16 or fp32 [width]) is added to with
    `accumulate`."""
    dev = _device(dy, "dy")
    pd, rows, width, sd = _matrix(dy, "dy", dev)
    shape, dtype = dy.shape, dy.dtype
    if dx is None:
        raise ValueError("dx is needed")
    po, so = _like(dx, shape, rows, width, dtype, "dx", dev)
    pe, se = _like(dh, shape, rows, width, dtype, "dh", dev)
    ph = sh = 0
    ref = None
    if isinstance(h, torch.Tensor):
        ph, sh = _like(h, shape, rows, width, dtype, "h", dev)
    else:
        ref = ctypes.byref(_checkpoint_arg(h, "h", rows, width, dev))
    if rstd is None:
        raise ValueError("rstd of the forward pass is needed")
    nbytes = _workspace_bytes("dpr_rmsnorm_backward_workspace", rows, width)
    handle = _handle(stream, dev)
    ws = _workspace(workspace, nbytes, stream, handle, dev)
    st = lib().dpr_rmsnorm_backward(
        pd, sd, pe, se, ph, sh, ref, rows, width, _code(dy, "dy"),
        _vector(weight, width, "weight", dev), 0 if weight is None else _code(weight, "weight"),
        _statistic(rstd, rows, "rstd", dev), po, so, _vector(dweight, width, "dweight", dev),
        0 if dweight is None else _code(dweight, "dweight"), 1 if accumulate else 0,
        0 if ws is None else ws.data_ptr(), nbytes, handle)
    if st:
        _check("dpr_rmsnorm_backward", st)


def _needed(t, what: str):
    if t is None:
        raise ValueError(f"{what}: a tensor is needed")


def _experts(t: torch.Tensor, what: str, dev: int):
    """(address, experts, rows, width, row stride, expert stride) of [experts, rows, width]."""
    _needed(t, what)
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
    _needed(t, "offsets")
    if t.dtype != torch.int32:
        raise ValueError(f"offsets: need torch.int32, got {t.dtype}")
    return _vector(t, experts + 1, "offsets", dev)


def _grouped_product(fn: str, x, what: str, offsets, weight, out, out_what: str, workspace, stream):
    """The product and its input gradient, which differ in the side of the
    weight that their argument and their result have."""
    dev = _device(x, what)
    px, rows, width, sx = _matrix(x, what, dev)
    _bf16(x, what)
    _needed(weight, "weight")
    _needed(out, out_what)
    _bf16(weight, "weight")
    pw, experts, o, i, sw, ew = _experts(weight, "weight", dev)
    have, give = (i, o) if fn == "dpr_grouped_linear" else (o, i)
    if width != have:
        raise ValueError(f"{what}: rows of {width}, but weight is {tuple(weight.shape)}")
    po, r, w, so = _matrix(out, out_what, dev)
    if r != rows or w != give:
        _wrong_shape(out_what, r, w, rows, give)
    offs = _offsets(offsets, experts, dev)
    # of the addresses only their alignment counts
    nbytes = _workspace_bytes(fn + "_workspace", px & 15, sx, rows, experts, pw & 15, sw, ew, o, i)
    handle = _handle(stream, dev)
    ws = _workspace(workspace, nbytes, stream, handle, dev)
    st = getattr(lib(), fn)(px, sx, rows, offs, experts, pw, sw, ew, o, i, po, so, _code(out, out_what),
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
        layout = (px & 15, sx)
    else:
        c = _checkpoint_arg(x, "x", rows, in_features, dev)
        ref = ctypes.byref(c)
        layout = ((c.codes or 0) & 15, c.code_stride, (c.steps or 0) & 15, c.step_stride)
    offs = _offsets(offsets, experts, dev)
    nbytes = _weight_grad_bytes(pd & 15, sd, layout, rows, experts, out_features, in_features)
    handle = _handle(stream, dev)
    ws = _workspace(workspace, nbytes, stream, handle, dev)
    st = lib().dpr_grouped_linear_weight_grad(
        pd, sd, px, sx, ref, rows, offs, experts, out_features, in_features, pw, sw, ew,
        _code(dweight, "dweight"), 1 if accumulate else 0, 0 if ws is None else ws.data_ptr(),
        nbytes, handle)
    if st:
        _check("dpr_grouped_linear_weight_grad", st)


@functools.lru_cache(maxsize=1024)
def _weight_grad_bytes(dy: int, dy_stride: int, x: tuple, rows: int, experts: int, out_features: int,
                       in_features: int) -> int:
    """Scratch memory by sizes and strides; of the addresses only their alignment counts."""
    px, sx, ref = x[0], x[1], None
    if len(x) == 4:
        px = sx = 0
        ref = ctypes.byref(_CheckpointArg(*x))
    n = ctypes.c_int64()
    _check("dpr_grouped_linear_weight_grad",
           lib().dpr_grouped_linear_weight_grad_workspace(dy, dy_stride, px, sx, ref, rows, experts,
                                                          out_features, in_features, ctypes.byref(n)))
    return n.value


class GradPlan:
    """Owns a dpr_grad_plan and keeps its tensors alive.  Keep it as long as the steps and
    the graphs captured with it: closing it frees device memory, which may wait for all of
    the device's work and must not happen while a stream is captured."""

    def __init__(self, handle: int, device: int, workspace_bytes: int, tensors: tuple):
        self.handle = handle
        self.device = device
        self.workspace_bytes = workspace_bytes
        self._tensors = tensors

    def close(self):
        if self.handle:
            h, self.handle = self.handle, None
            _check("dpr_grad_plan_destroy", lib().dpr_grad_plan_destroy(h))

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _dtypes(ts: Sequence[torch.Tensor], what: str, dev: int):
    """Type codes of contiguous tensors on the current device."""
    codes = (ctypes.c_int * len(ts))()
    for i, t in enumerate(ts):
        if t.get_device() != dev:
            _wrong_device(t, what)
        c = _DTYPES.get(t.dtype)
        if c is None or not t.is_contiguous():
            raise ValueError(f"{what}: need contiguous torch.bfloat16 or torch.float32 tensors")
        codes[i] = c
    return codes


def dpr_grad_plan_create(grads: Sequence[torch.Tensor], outs=None, stream=None) -> GradPlan:
    """A list of gradients (contiguous, bf16 or fp32, any shapes) whose norm is
    taken and that are clipped into `outs` (as many elements each, bf16 or
    fp32; without it, in place)."""
    grads = list(grads)
    n = len(grads)
    dev = _device(grads[0], "grads") if n else torch.cuda.current_device()
    src = _dtypes(grads, "grads", dev)
    numel = (ctypes.c_int64 * n)(*[t.numel() for t in grads])
    dst = to = None
    if outs is not None:
        outs = list(outs)
        if len(outs) != n:
            raise ValueError(f"outs: expected {n} tensors, got {len(outs)}")
        to = _dtypes(outs, "outs", dev)
        for g, o in zip(grads, outs):
            if o.numel() != g.numel():
                raise ValueError(f"outs: need {g.numel()} elements, got {o.numel()}")
        dst = _ptrs(outs)
    h = ctypes.c_void_p()
    _check("dpr_grad_plan_create",
           lib().dpr_grad_plan_create(ctypes.byref(h), n, _ptrs(grads), src, dst, to, numel,
                                      _stream(stream)))
    nbytes = ctypes.c_int64()
    plan = GradPlan(h.value, dev, 0, (grads, outs))
    _check("dpr_grad_norm_workspace", lib().dpr_grad_norm_workspace(h, ctypes.byref(nbytes)))
    plan.workspace_bytes = nbytes.value
    return plan


def dpr_grad_plan_destroy(plan: GradPlan) -> None:
    plan.close()


def _norm(plan: GradPlan, norm: torch.Tensor) -> int:
    if plan.handle is None:
        raise ValueError("the plan is closed")
    _needed(norm, "norm")
    dev = _device(norm, "norm")
    if dev != plan.device:
        raise ValueError(f"the plan's tensors are on cuda:{plan.device}, norm is on cuda:{dev}")
    return _statistic(norm, 1, "norm", dev)


def dpr_grad_norm(plan: GradPlan, norm: torch.Tensor, scale: float = 1.0, workspace=None,
                  stream=None) -> None:
    """norm (one fp32 number on the device) = scale * sqrt(sum of squares of all
    elements of the plan's gradients)."""
    pn = _norm(plan, norm)
    handle = _handle(stream, plan.device)
    ws = _workspace(workspace, plan.workspace_bytes, stream, handle, plan.device)
    st = lib().dpr_grad_norm(plan.handle, scale, pn, 0 if ws is None else ws.data_ptr(),
                             plan.workspace_bytes, handle)
    if st:
        _check("dpr_grad_norm", st)


def dpr_grad_clip(plan: GradPlan, norm: torch.Tensor, max_norm: float, scale: float = 1.0,
                  stream=None) -> None:
    """Every gradient times scale, and times max_norm / norm where norm is larger
    than max_norm; `norm` as dpr_grad_norm leaves it, or joined with others'."""
    pn = _norm(plan, norm)
    st = lib().dpr_grad_clip(plan.handle, scale, max_norm, pn, _handle(stream, plan.device))
    if st:
        _check("dpr_grad_clip", st)


def dpr_grad_norm_clip(plan: GradPlan, norm: torch.Tensor, max_norm: float, scale: float = 1.0,
                       workspace=None, stream=None) -> None:
    """dpr_grad_norm and dpr_grad_clip in one call."""
    pn = _norm(plan, norm)
    handle = _handle(stream, plan.device)
    ws = _workspace(workspace, plan.workspace_bytes, stream, handle, plan.device)
    st = lib().dpr_grad_norm_clip(plan.handle, scale, max_norm, pn,
                                  0 if ws is None else ws.data_ptr(), plan.workspace_bytes, handle)
    if st:
        _check("dpr_grad_norm_clip", st)
