"""Binding of the backward-pass operators (include/dpr_ops.h): layer norm,
8-bit activation checkpoints and the weight gradient read from them.

Activations are tensors [..., width] whose last dimension is contiguous and
whose leading dimensions merge into one row stride without a copy.  As in
the rest of the package, the checks here keep a wrongly shaped, typed or
placed tensor from being read or written out of bounds; libdpr checks
strides, alignment and overlap, and does all of the computing.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import _check, _stream, lib

CHECKPOINT_BLOCK = 32            # channels that share a step
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


class _CheckpointArg(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("code_stride", ctypes.c_int64),
                ("steps", ctypes.c_void_p), ("step_stride", ctypes.c_int64)]


class Checkpoint:
    """An activation held in 8 bits: `codes` int8 [rows, width] and `steps`
    uint8 [rows, ceil(width / 32)], views of any row stride.  Row strides and
    addresses that are multiples of 16 bytes, as dpr_checkpoint_empty lays
    them out, take the fastest kernels."""

    __slots__ = ("codes", "steps")

    def __init__(self, codes: torch.Tensor, steps: torch.Tensor):
        self.codes, self.steps = codes, steps

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.steps.numel()


def dpr_checkpoint_empty(rows: int, width: int, device=None) -> Checkpoint:
    """Room for an activation of `rows` x `width`, rows padded to 16 bytes."""
    blocks = -(-width // CHECKPOINT_BLOCK)
    device = "cuda" if device is None else device
    codes = torch.empty(rows, -(-width // 16) * 16, dtype=torch.int8, device=device)
    steps = torch.empty(rows, -(-blocks // 16) * 16, dtype=torch.uint8, device=device)
    return Checkpoint(codes[:, :width], steps[:, :blocks])


def _on_device(t: torch.Tensor, what: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{what}: need a CUDA tensor")
    dev = torch.cuda.current_device()
    if t.get_device() != dev:
        raise ValueError(f"{what}: tensor on cuda:{t.get_device()}, current device is cuda:{dev}")


def _matrix(t: torch.Tensor, what: str, dtypes=_DTYPES):
    """(address, rows, width, row stride) of a tensor as a matrix."""
    _on_device(t, what)
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: {t.dtype} is not among {', '.join(map(str, dtypes))}")
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError(f"{what}: need at least one dimension")
        try:
            t = t.view(-1, t.shape[-1]) if t.numel() else t.new_empty(
                (t.shape[:-1].numel(), t.shape[-1]))
        except RuntimeError:
            raise ValueError(f"{what}: the leading dimensions do not merge into one row stride, "
                             f"shape {tuple(t.shape)} strides {t.stride()}") from None
    rows, width = t.shape
    stride, inner = t.stride()
    if width > 1 and inner != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr(), rows, width, stride if rows > 1 else max(stride, width)


def _same(what: str, got, want) -> None:
    if tuple(got) != tuple(want):
        raise ValueError(f"{what}: need {want[0]} rows of {want[1]}, got {got[0]} of {got[1]}")


def _checkpoint_arg(c, what: str):
    """(C struct, rows, width) of a Checkpoint."""
    if not isinstance(c, Checkpoint):
        raise ValueError(f"{what}: need a Checkpoint, got {type(c).__name__}")
    pc, rows, width, sc = _matrix(c.codes, what + ".codes", (torch.int8,))
    ps, srows, blocks, ss = _matrix(c.steps, what + ".steps", (torch.uint8,))
    if srows != rows or blocks < -(-width // CHECKPOINT_BLOCK):
        raise ValueError(f"{what}: {rows} rows of {width} codes need as many rows of "
                         f"{-(-width // CHECKPOINT_BLOCK)} steps, got {srows} of {blocks}")
    return _CheckpointArg(pc, sc, ps, ss), rows, width


def _vector(t, n: int, what: str, dtypes=_DTYPES):
    """Address of a contiguous vector of n elements; 0 for None."""
    if t is None:
        return 0
    _on_device(t, what)
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: {t.dtype} is not among {', '.join(map(str, dtypes))}")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: need {n} contiguous elements")
    return t.data_ptr()


_FP32 = (torch.float32,)


def _pair_dtype(a, b, what: str) -> int:
    """The common type code of two optional tensors."""
    if a is None and b is None:
        return 0
    if a is not None and b is not None and a.dtype != b.dtype:
        raise ValueError(f"{what} must have one dtype, got {a.dtype} and {b.dtype}")
    return _DTYPES[(b if a is None else a).dtype]


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(fn: str, *sizes: int) -> int:
    n = ctypes.c_int64()
    _check(fn, getattr(lib(), fn)(*sizes, ctypes.byref(n)))
    return n.value


def _workspace(t, nbytes: int, stream):
    """The caller's scratch memory, or some from PyTorch's allocator, taken on
    the stream that uses it so that it is not handed out again too early."""
    if t is not None:
        _on_device(t, "workspace")
        if not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
            raise ValueError(f"workspace: need {nbytes} contiguous bytes")
        return t
    if nbytes == 0:
        return None
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def dpr_layernorm_forward(x: torch.Tensor, weight, bias, eps: float, y: torch.Tensor, mean=None,
                          rstd=None, x_checkpoint=None, y_checkpoint=None, stream=None) -> None:
    """y = (x - mean) * rstd * weight + bias along the last dimension; weight
    and bias (bf16 or fp32) may be None.  mean and rstd ([rows] fp32) are what
    the backward pass needs.  The checkpoints, where given, are written in
    the same pass as dpr_checkpoint_save(x) and (y) would.  y may be x."""
    px, rows, width, sx = _matrix(x, "x")
    py, *shape, sy = _matrix(y, "y")
    _same("y", shape, (rows, width))
    if y.dtype != x.dtype:
        raise ValueError(f"y: {y.dtype}, but x is {x.dtype}")
    refs = []
    for c, what in ((x_checkpoint, "x_checkpoint"), (y_checkpoint, "y_checkpoint")):
        if c is None:
            refs.append(None)
            continue
        arg, *shape = _checkpoint_arg(c, what)
        _same(what, shape, (rows, width))
        refs.append(ctypes.byref(arg))
    st = lib().dpr_layernorm_forward(
        px, sx, rows, width, _DTYPES[x.dtype], _vector(weight, width, "weight"),
        _vector(bias, width, "bias"), _pair_dtype(weight, bias, "weight and bias"), eps, py, sy,
        _vector(mean, rows, "mean", _FP32), _vector(rstd, rows, "rstd", _FP32), refs[0], refs[1],
        _stream(stream))
    _check("dpr_layernorm_forward", st)


def dpr_layernorm_backward(dy: torch.Tensor, x, weight, mean: torch.Tensor, rstd: torch.Tensor,
                           dx: torch.Tensor, dweight=None, dbias=None, accumulate: bool = False,
                           workspace=None, stream=None) -> None:
    """dx, dweight and dbias of dpr_layernorm_forward.  `x` is the forward's
    input or its Checkpoint.  dweight and dbias (bf16 or fp32 [width], None
    where not wanted) are added to with `accumulate`.  dx may be dy or x."""
    pd, rows, width, sd = _matrix(dy, "dy")
    po, *shape, so = _matrix(dx, "dx")
    _same("dx", shape, (rows, width))
    if dx.dtype != dy.dtype:
        raise ValueError(f"dx: {dx.dtype}, but dy is {dy.dtype}")
    px = sx = 0
    ref = None
    if isinstance(x, torch.Tensor):
        px, *shape, sx = _matrix(x, "x")
        if x.dtype != dy.dtype:
            raise ValueError(f"x: {x.dtype}, but dy is {dy.dtype}")
    else:
        arg, *shape = _checkpoint_arg(x, "x")
        ref = ctypes.byref(arg)
    _same("x", shape, (rows, width))
    if mean is None or rstd is None:
        raise ValueError("mean and rstd of the forward pass are needed")
    nbytes = _workspace_bytes("dpr_layernorm_backward_workspace", rows, width)
    ws = _workspace(workspace, nbytes, stream)
    st = lib().dpr_layernorm_backward(
        pd, sd, px, sx, ref, rows, width, _DTYPES[dy.dtype], _vector(weight, width, "weight"),
        0 if weight is None else _DTYPES[weight.dtype], _vector(mean, rows, "mean", _FP32),
        _vector(rstd, rows, "rstd", _FP32), po, so, _vector(dweight, width, "dweight"),
        _vector(dbias, width, "dbias"), _pair_dtype(dweight, dbias, "dweight and dbias"),
        int(bool(accumulate)), 0 if ws is None else ws.data_ptr(), nbytes, _stream(stream))
    _check("dpr_layernorm_backward", st)


def dpr_checkpoint_save(x: torch.Tensor, checkpoint: Checkpoint, stream=None) -> None:
    """Saves x ([..., width] bf16 or fp32) in 8 bits."""
    px, rows, width, sx = _matrix(x, "x")
    arg, *shape = _checkpoint_arg(checkpoint, "checkpoint")
    _same("checkpoint", shape, (rows, width))
    _check("dpr_checkpoint_save", lib().dpr_checkpoint_save(
        px, sx, rows, width, _DTYPES[x.dtype], ctypes.byref(arg), _stream(stream)))


def dpr_checkpoint_load(checkpoint: Checkpoint, out: torch.Tensor, stream=None) -> None:
    """Restores a checkpoint into out ([..., width] bf16 or fp32)."""
    po, rows, width, so = _matrix(out, "out")
    arg, *shape = _checkpoint_arg(checkpoint, "checkpoint")
    _same("checkpoint", shape, (rows, width))
    _check("dpr_checkpoint_load", lib().dpr_checkpoint_load(
        ctypes.byref(arg), rows, width, po, so, _DTYPES[out.dtype], _stream(stream)))


def dpr_linear_weight_grad(dy: torch.Tensor, x_checkpoint: Checkpoint, dweight: torch.Tensor,
                           accumulate: bool = False, workspace=None, stream=None) -> None:
    """dweight = dy^T x with dy bf16 [..., out_features] and the checkpoint
    of x [rows, in_features]; dweight bf16 or fp32 [out_features,
    in_features], added to with `accumulate`."""
    pd, rows, out_features, sd = _matrix(dy, "dy", (torch.bfloat16,))
    arg, xrows, in_features = _checkpoint_arg(x_checkpoint, "x_checkpoint")
    if xrows != rows:
        raise ValueError(f"x_checkpoint: {xrows} rows, but dy has {rows}")
    if dweight.dim() != 2:
        raise ValueError("dweight: need a matrix")
    pw, *shape, sw = _matrix(dweight, "dweight")
    _same("dweight", shape, (out_features, in_features))
    ref = ctypes.byref(arg)
    need = ctypes.c_int64()
    _check("dpr_linear_weight_grad", lib().dpr_linear_weight_grad_workspace(
        pd, sd, ref, rows, out_features, in_features, ctypes.byref(need)))
    nbytes = need.value
    ws = _workspace(workspace, nbytes, stream)
    _check("dpr_linear_weight_grad", lib().dpr_linear_weight_grad(
        pd, sd, ref, rows, out_features, in_features, pw, sw, _DTYPES[dweight.dtype],
        int(bool(accumulate)), 0 if ws is None else ws.data_ptr(), nbytes, _stream(stream)))


def dpr_device_wait_failures() -> int:
    """Waits inside the weight gradient's kernel that have run out (0 in
    working order); waits for the device."""
    n = ctypes.c_uint32()
    _check("dpr_device_wait_failures", lib().dpr_device_wait_failures(ctypes.byref(n)))
    return n.value
