"""Binding of the backward-pass operators (include/dpr_ops.h): layer norm,
8-bit activation checkpoints and the weight gradient read from them.

Activations are tensors [..., width] whose last dimension is contiguous and
whose leading dimensions merge into one row stride without a copy.  As in
the rest of the package, the checks here keep a wrongly shaped, typed or
placed tensor from being read or written out of bounds; libdpr checks
strides, alignment and overlap, and does all of the computing.

Calls that need scratch memory take it as `workspace`.  Without one they use
PyTorch's: on the current stream memory that is kept from call to call, for
each thread and stream the most that a call asked for (up to 64 MiB; larger
sizes are allocated per call), until the thread ends.  It is known by the
stream's handle, so a stream made outside PyTorch has to be idle when it is
destroyed, as PyTorch's own memory on it demands.
"""
from __future__ import annotations

import ctypes
import functools
import threading

import torch

from ._binding import _check, _raw_stream, _stream, lib

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


def _wrong_device(t: torch.Tensor, what: str):
    if not t.is_cuda:
        raise ValueError(f"{what}: need a CUDA tensor")
    raise ValueError(f"{what}: tensor on cuda:{t.get_device()}, current device is "
                     f"cuda:{torch.cuda.current_device()}")


# The current device without torch.cuda.current_device()'s lazy initialisation
# checks (0.3 us a call); a CUDA tensor at hand means that CUDA is up.
_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device(t: torch.Tensor, what: str) -> int:
    """The current device, on which the call's tensors have to be: the kernels
    would fault on another's memory."""
    dev = t.get_device()
    if dev < 0 or dev != _get_device():
        _wrong_device(t, what)
    return dev


def _handle(stream, dev: int) -> int:
    """The handle of `stream`; without one, of the current device's current stream."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(dev)
    return _stream(stream)


def _matrix(t: torch.Tensor, what: str, dev: int):
    """(address, rows, width, row stride) of a tensor as a matrix."""
    if t.get_device() != dev:
        _wrong_device(t, what)
    if t.dim() != 2:
        t = _merge(t, what)
    rows, width = t.shape
    stride, inner = t.stride()
    if inner != 1 and width > 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return t.data_ptr(), rows, width, stride if rows > 1 or stride > width else width


def _merge(t: torch.Tensor, what: str) -> torch.Tensor:
    if t.dim() == 0:
        raise ValueError(f"{what}: need at least one dimension")
    if t.numel() == 0:
        return t.new_empty((t.shape[:-1].numel(), t.shape[-1]))
    try:
        return t.view(-1, t.shape[-1])
    except RuntimeError:
        raise ValueError(f"{what}: the leading dimensions do not merge into one row stride, "
                         f"shape {tuple(t.shape)} strides {t.stride()}") from None


def _code(t: torch.Tensor, what: str) -> int:
    """The type code of a bf16 or fp32 tensor."""
    c = _DTYPES.get(t.dtype)
    if c is None:
        raise ValueError(f"{what}: {t.dtype} is neither torch.bfloat16 nor torch.float32")
    return c


def _checkpoint_arg(c, what: str, rows: int, width: int, dev: int):
    """The C struct of a Checkpoint of `rows` x `width`."""
    if not isinstance(c, Checkpoint):
        raise ValueError(f"{what}: need a Checkpoint, got {type(c).__name__}")
    codes, steps = c.codes, c.steps
    if codes.dtype != torch.int8 or steps.dtype != torch.uint8:
        raise ValueError(f"{what}: need int8 codes and uint8 steps, got {codes.dtype} and {steps.dtype}")
    pc, r, w, sc = _matrix(codes, what, dev)
    ps, sr, blocks, ss = _matrix(steps, what, dev)
    if r != rows or w != width:
        _wrong_shape(what, r, w, rows, width)
    if sr != rows or blocks * CHECKPOINT_BLOCK < width:
        raise ValueError(f"{what}: {rows} rows of {width} codes need as many rows of "
                         f"{-(-width // CHECKPOINT_BLOCK)} steps, got {sr} of {blocks}")
    return _CheckpointArg(pc, sc, ps, ss)


def _wrong_shape(what: str, rows: int, width: int, want_rows: int, want_width: int):
    raise ValueError(f"{what}: need {want_rows} rows of {want_width}, got {rows} of {width}")


def _vector(t, n: int, what: str, dev: int) -> int:
    """Address of a contiguous vector of n elements; 0 for None."""
    if t is None:
        return 0
    if t.get_device() != dev:
        _wrong_device(t, what)
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: need {n} contiguous elements")
    return t.data_ptr()


def _statistic(t, n: int, what: str, dev: int) -> int:
    if t is not None and t.dtype != torch.float32:
        raise ValueError(f"{what}: need torch.float32, got {t.dtype}")
    return _vector(t, n, what, dev)


def _pair_code(a, b, what: str) -> int:
    """The common type code of two optional tensors."""
    if a is None:
        return 0 if b is None else _code(b, what)
    if b is not None and a.dtype != b.dtype:
        raise ValueError(f"{what} must have one dtype, got {a.dtype} and {b.dtype}")
    return _code(a, what)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(fn: str, *sizes: int) -> int:
    n = ctypes.c_int64()
    _check(fn, getattr(lib(), fn)(*sizes, ctypes.byref(n)))
    return n.value


class _Scratch(threading.local):
    """Scratch memory kept between calls, per thread and stream: the calls of
    one stream run in order, so they may share it, and a thread's calls are
    enqueued whole.  (An allocation per call cost 6 to 8 us of host time.)"""

    def __init__(self):
        self.kept = {}


_scratch = _Scratch()
_KEEP_BYTES = 64 << 20
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing",
                     torch.cuda.is_current_stream_capturing)


def _workspace(t, nbytes: int, stream, handle: int, dev: int):
    """The caller's scratch memory, or some of PyTorch's: kept between calls on
    the current stream, except inside a graph capture, whose memory has to be
    the graph's own.  For another stream it is allocated there, so that it is
    not handed out again before that stream is done with it."""
    if t is not None:
        if t.get_device() != dev:
            _wrong_device(t, "workspace")
        if not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
            raise ValueError(f"workspace: need {nbytes} contiguous bytes")
        return t
    if nbytes == 0:
        return None
    if stream is None:
        if nbytes > _KEEP_BYTES or _capturing():
            return torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        key = (dev, handle)
        t = _scratch.kept.get(key)
        if t is None or t.numel() < nbytes:
            t = _scratch.kept[key] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        return t
    if not isinstance(stream, torch.cuda.Stream):
        # 0 and 1 (cudaStreamLegacy) are the default stream; ExternalStream makes a new
        # stream of PyTorch's pool of 0, and memory freed there would be handed out again
        # while the default stream still uses it, and takes no 1
        stream = (torch.cuda.default_stream(dev) if int(stream) in (0, 1)
                  else torch.cuda.ExternalStream(int(stream)))
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device="cuda")


def dpr_layernorm_forward(x: torch.Tensor, weight, bias, eps: float, y: torch.Tensor, mean=None,
                          rstd=None, x_checkpoint=None, y_checkpoint=None, stream=None) -> None:
    """y = (x - mean) * rstd * weight + bias along the last dimension; weight
    and bias (bf16 or fp32) may be None.  mean and rstd ([rows] fp32) are what
    the backward pass needs.  The checkpoints, where given, are written in
    the same pass as dpr_checkpoint_save(x) and (y) would.  y may be x."""
    dev = _device(x, "x")
    px, rows, width, sx = _matrix(x, "x", dev)
    py, r, w, sy = _matrix(y, "y", dev)
    if r != rows or w != width:
        _wrong_shape("y", r, w, rows, width)
    if y.dtype != x.dtype:
        raise ValueError(f"y: {y.dtype}, but x is {x.dtype}")
    cx = cy = None
    if x_checkpoint is not None:
        cx = ctypes.byref(_checkpoint_arg(x_checkpoint, "x_checkpoint", rows, width, dev))
    if y_checkpoint is not None:
        cy = ctypes.byref(_checkpoint_arg(y_checkpoint, "y_checkpoint", rows, width, dev))
    st = lib().dpr_layernorm_forward(
        px, sx, rows, width, _code(x, "x"), _vector(weight, width, "weight", dev),
        _vector(bias, width, "bias", dev), _pair_code(weight, bias, "weight and bias"), eps, py, sy,
        _statistic(mean, rows, "mean", dev), _statistic(rstd, rows, "rstd", dev), cx, cy,
        _handle(stream, dev))
    if st:
        _check("dpr_layernorm_forward", st)


def dpr_layernorm_backward(dy: torch.Tensor, x, weight, mean: torch.Tensor, rstd: torch.Tensor,
                           dx: torch.Tensor, dweight=None, dbias=None, accumulate: bool = False,
                           workspace=None, stream=None) -> None:
    """dx, dweight and dbias of dpr_layernorm_forward.  `x` is the forward's
    input or its Checkpoint.  dweight and dbias (bf16 or fp32 [width], None
    where not wanted) are added to with `accumulate`.  dx may be dy or x."""
    dev = _device(dy, "dy")
    pd, rows, width, sd = _matrix(dy, "dy", dev)
    po, r, w, so = _matrix(dx, "dx", dev)
    if r != rows or w != width:
        _wrong_shape("dx", r, w, rows, width)
    if dx.dtype != dy.dtype:
        raise ValueError(f"dx: {dx.dtype}, but dy is {dy.dtype}")
    px = sx = 0
    ref = None
    if isinstance(x, torch.Tensor):
        px, r, w, sx = _matrix(x, "x", dev)
        if r != rows or w != width:
            _wrong_shape("x", r, w, rows, width)
        if x.dtype != dy.dtype:
            raise ValueError(f"x: {x.dtype}, but dy is {dy.dtype}")
    else:
        ref = ctypes.byref(_checkpoint_arg(x, "x", rows, width, dev))
    if mean is None or rstd is None:
        raise ValueError("mean and rstd of the forward pass are needed")
    nbytes = _workspace_bytes("dpr_layernorm_backward_workspace", rows, width)
    handle = _handle(stream, dev)
    ws = _workspace(workspace, nbytes, stream, handle, dev)
    st = lib().dpr_layernorm_backward(
        pd, sd, px, sx, ref, rows, width, _code(dy, "dy"), _vector(weight, width, "weight", dev),
        0 if weight is None else _code(weight, "weight"), _statistic(mean, rows, "mean", dev),
        _statistic(rstd, rows, "rstd", dev), po, so, _vector(dweight, width, "dweight", dev),
        _vector(dbias, width, "dbias", dev), _pair_code(dweight, dbias, "dweight and dbias"),
        1 if accumulate else 0, 0 if ws is None else ws.data_ptr(), nbytes, handle)
    if st:
        _check("dpr_layernorm_backward", st)


def dpr_checkpoint_save(x: torch.Tensor, checkpoint: Checkpoint, stream=None) -> None:
    """Saves x ([..., width] bf16 or fp32) in 8 bits."""
    dev = _device(x, "x")
    px, rows, width, sx = _matrix(x, "x", dev)
    arg = _checkpoint_arg(checkpoint, "checkpoint", rows, width, dev)
    st = lib().dpr_checkpoint_save(px, sx, rows, width, _code(x, "x"), ctypes.byref(arg),
                                   _handle(stream, dev))
    if st:
        _check("dpr_checkpoint_save", st)


def dpr_checkpoint_load(checkpoint: Checkpoint, out: torch.Tensor, stream=None) -> None:
    """Restores a checkpoint into out ([..., width] bf16 or fp32)."""
    dev = _device(out, "out")
    po, rows, width, so = _matrix(out, "out", dev)
    arg = _checkpoint_arg(checkpoint, "checkpoint", rows, width, dev)
    st = lib().dpr_checkpoint_load(ctypes.byref(arg), rows, width, po, so, _code(out, "out"),
                                   _handle(stream, dev))
    if st:
        _check("dpr_checkpoint_load", st)


def dpr_linear_weight_grad(dy: torch.Tensor, x_checkpoint: Checkpoint, dweight: torch.Tensor,
                           accumulate: bool = False, workspace=None, stream=None) -> None:
    """dweight = dy^T x with dy bf16 [..., out_features] and the checkpoint
    of x [rows, in_features]; dweight bf16 or fp32 [out_features,
    in_features], added to with `accumulate`."""
    dev = _device(dy, "dy")
    pd, rows, out_features, sd = _matrix(dy, "dy", dev)
    if dy.dtype != torch.bfloat16:
        raise ValueError(f"dy: need torch.bfloat16, got {dy.dtype}")
    if dweight.dim() != 2:
        raise ValueError("dweight: need a matrix")
    pw, r, in_features, sw = _matrix(dweight, "dweight", dev)
    if r != out_features:
        raise ValueError(f"dweight: {r} rows, but dy has {out_features} out-features")
    ref = ctypes.byref(_checkpoint_arg(x_checkpoint, "x_checkpoint", rows, in_features, dev))
    need = ctypes.c_int64()
    L = lib()
    st = L.dpr_linear_weight_grad_workspace(pd, sd, ref, rows, out_features, in_features,
                                            ctypes.byref(need))
    if st:
        _check("dpr_linear_weight_grad", st)
    nbytes = need.value
    handle = _handle(stream, dev)
    ws = _workspace(workspace, nbytes, stream, handle, dev)
    st = L.dpr_linear_weight_grad(
        pd, sd, ref, rows, out_features, in_features, pw, sw, _code(dweight, "dweight"),
        1 if accumulate else 0, 0 if ws is None else ws.data_ptr(), nbytes, handle)
    if st:
        _check("dpr_linear_weight_grad", st)


def dpr_device_wait_failures() -> int:
    """How often a wait inside the operators' kernels has run out (0 in working
    order); waits for all of the device's work, on every stream."""
    n = ctypes.c_uint32()
    _check("dpr_device_wait_failures", lib().dpr_device_wait_failures(ctypes.byref(n)))
    return n.value
