"""Python binding of the C ABI in include/gdn_stack.h: what a stack needs between its layers and at
its end.

Argument marshalling only, as in api.py.  Rows may be a stride apart (views of a wider tensor); the
elements of a row are contiguous.
"""

from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from . import _lib
from .api import _DTYPES, _ptr


@dataclasses.dataclass(frozen=True)
class NormShape:
    """group: columns to a scale of the 8-bit output (128), 0 for one scale to a row, -1 for no such output."""

    width: int
    dtype: torch.dtype = torch.bfloat16
    residual_dtype: Optional[torch.dtype] = None  # None: dtype
    group: int = -1
    eps: float = 1e-6
    zero_centered: bool = False

    def __post_init__(self):
        if self.residual_dtype is None:
            object.__setattr__(self, "residual_dtype", self.dtype)
        for t in (self.dtype, self.residual_dtype):
            if t not in _DTYPES:
                raise ValueError(f"unsupported dtype {t}")
        object.__setattr__(self, "_ref", ctypes.byref(_lib.NormShapeC(
            self.width, _DTYPES[self.dtype], _DTYPES[self.residual_dtype], self.group, self.zero_centered, self.eps)))

    def __reduce__(self):
        return NormShape, tuple(getattr(self, f.name) for f in dataclasses.fields(self))


@dataclasses.dataclass(frozen=True)
class LogitsShape:
    """top: the alternatives to a row that gdn_stack_logprobs gives, or the teacher's entries to a row
    that gdn_stack_distill takes, whose values are log probabilities if teacher_logprobs is set."""

    vocab: int
    dtype: torch.dtype = torch.bfloat16
    top: int = 0
    teacher_logprobs: bool = False

    def __post_init__(self):
        if self.dtype not in _DTYPES:
            raise ValueError(f"unsupported dtype {self.dtype}")
        object.__setattr__(self, "_ref", ctypes.byref(_lib.LogitsShapeC(self.vocab, _DTYPES[self.dtype], self.top,
                                                                       self.teacher_logprobs)))

    def __reduce__(self):
        return LogitsShape, tuple(getattr(self, f.name) for f in dataclasses.fields(self))


def gdn_stack_norm_workspace_size(shape: NormShape, rows: int) -> int:
    return int(_lib.load().gdn_stack_norm_workspace_size(shape._ref, rows))


def gdn_stack_logits_workspace_size(shape: LogitsShape, rows: int) -> int:
    return int(_lib.load().gdn_stack_logits_workspace_size(shape._ref, rows))


def alloc_norm_workspace(shape: NormShape, rows: int, device="cuda") -> torch.Tensor:
    """For gdn_stack_add_norm_bwd."""
    return torch.empty(max(gdn_stack_norm_workspace_size(shape, rows), 256), dtype=torch.uint8, device=device)


def alloc_logits_workspace(shape: LogitsShape, rows: int, device="cuda") -> torch.Tensor:
    """For gdn_stack_logprobs and gdn_stack_distill (their gradients need none)."""
    return torch.empty(max(gdn_stack_logits_workspace_size(shape, rows), 256), dtype=torch.uint8, device=device)


def _row_args(t, rows, width: int, dtype, name: str):
    """(rows, pointer, row stride) of a [rows, width] tensor whose rows are contiguous; a given
    number of rows is checked.  None: (rows, None, 0)."""
    if t is None:
        return rows, None, 0
    shape = t.shape
    if len(shape) != 2 or shape[1] != width or t.dtype is not dtype or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name}: [{'rows' if rows is None else rows}, {width}] of {dtype} expected, "
                         f"{tuple(shape)} of {t.dtype} given")
    n = shape[0]
    if t.is_contiguous():  # the usual case, and a fifth cheaper than to ask for the strides
        return n, t.data_ptr(), 0
    s0, s1 = t.stride()
    if width > 1 and s1 != 1:
        raise ValueError(f"{name}: a row's elements must be contiguous")
    if n > 1 and s0 < width:
        raise ValueError(f"{name}: rows overlap")
    return n, t.data_ptr(), s0 if n > 1 else 0


def _whole(t, shape: tuple, dtype, name: str):
    """Pointer of a contiguous tensor of the given shape; None for None."""
    if t is None:
        return None
    if tuple(t.shape) != shape or t.dtype is not dtype or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {shape} of {dtype} expected, {tuple(t.shape)} of {t.dtype} given")
    return t.data_ptr()


def _weight(w, width: int, name: str):
    if w.dtype is not torch.float32 or w.numel() != width or not w.is_contiguous():
        raise ValueError(f"{name}: contiguous float32 of {width} expected")
    return w.data_ptr()


def _stream(stream, *tensors) -> int:
    """The handle of the stream, or of the current one; the tensors have to be on its device, and that
    has to be the current one."""
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != device or device < 0:
            raise ValueError(f"a tensor is on {t.device}, the first one on {tensors[0].device}")
    if device != torch.cuda.current_device():
        raise ValueError(f"the tensors are on cuda:{device}, which is not the current device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError(f"the stream is of cuda:{stream.device_index}, the tensors are on cuda:{device}")
    return stream.cuda_stream


def _bytes(workspace):
    if not workspace.is_contiguous():
        raise ValueError("workspace: contiguous expected")
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def gdn_stack_add_norm(shape: NormShape, x, residual, w, residual_out, y, y8=None, y_scale=None, stream=None) -> None:
    """residual_out = x + residual (residual None: x), y its norm, y8 and y_scale the norm in e4m3
    (uint8 codes) with scales; residual_out, and one of y and y8, may be None."""
    width, dt, rdt = shape.width, shape.dtype, shape.residual_dtype
    n, xp, xs = _row_args(x, None, width, dt, "x")
    _, rp, rs = _row_args(residual, n, width, rdt, "residual")
    _, hp, hs = _row_args(residual_out, n, width, rdt, "residual_out")
    _, yp, ys = _row_args(y, n, width, dt, "y")
    _lib.check(_lib.load().gdn_stack_add_norm(
        shape._ref, n, xp, xs, rp, rs, _weight(w, width, "w"), hp, hs, yp, ys, _whole(y8, (n, width), torch.uint8, "y8"),
        _whole(y_scale, (n, width // shape.group if shape.group > 0 else 1), torch.float32, "y_scale"),
        _stream(stream, x, residual, w, residual_out, y, y8, y_scale)))


def gdn_stack_add_norm_bwd(shape: NormShape, h, w, dy, d_residual_out, dx, d_residual, dw, workspace,
                           stream=None) -> None:
    """Gradients of gdn_stack_add_norm from h (its residual_out): dx in dtype and d_residual in
    residual_dtype, either may be None, and dw in fp32.  d_residual_out: the gradient that
    residual_out has from its other readers, or None."""
    width, dt, rdt = shape.width, shape.dtype, shape.residual_dtype
    n, hp, hs = _row_args(h, None, width, rdt, "h")
    _, yp, ys = _row_args(dy, n, width, dt, "dy")
    _, rp, rs = _row_args(d_residual_out, n, width, rdt, "d_residual_out")
    _, xp, xs = _row_args(dx, n, width, dt, "dx")
    _, dp, ds = _row_args(d_residual, n, width, rdt, "d_residual")
    _lib.check(_lib.load().gdn_stack_add_norm_bwd(
        shape._ref, n, hp, hs, _weight(w, width, "w"), yp, ys, rp, rs, xp, xs, dp, ds, _weight(dw, width, "dw"),
        *_bytes(workspace), _stream(stream, h, w, dy, d_residual_out, dx, d_residual, dw, workspace)))


def gdn_stack_logprobs(shape: LogitsShape, logits, targets, logprobs, entropy, top_ids, top_logprobs, stats, workspace,
                       scale=None, stream=None) -> None:
    """Log probabilities of the targets, the entropy and the top alternatives of every row of logits,
    and the statistics that the gradient takes.  Outputs that are not wanted are None; rows whose
    target is no index of the vocabulary are left out.  scale: one over the temperature, per row."""
    f32, i32, k = torch.float32, torch.int32, shape.top
    n, lp, ls = _row_args(logits, None, shape.vocab, shape.dtype, "logits")
    _lib.check(_lib.load().gdn_stack_logprobs(
        shape._ref, n, lp, ls, _whole(targets, (n,), i32, "targets"), _whole(scale, (n,), f32, "scale"),
        _whole(logprobs, (n,), f32, "logprobs"), _whole(entropy, (n,), f32, "entropy"),
        _whole(top_ids, (n, k), i32, "top_ids"), _whole(top_logprobs, (n, k), f32, "top_logprobs"),
        _whole(stats, (n, 2), f32, "stats"), *_bytes(workspace),
        _stream(stream, logits, targets, scale, logprobs, entropy, top_ids, top_logprobs, stats, workspace)))


def gdn_stack_logprobs_bwd(shape: LogitsShape, logits, targets, stats, entropy, d_logprobs, d_entropy, d_logits,
                           scale=None, stream=None) -> None:
    """Gradient of the log probabilities and the entropy; one of d_logprobs and d_entropy may be
    None (entropy with the latter).  targets are those of the forward call, with d_entropy alone too:
    they say which rows it left out.  d_logits may be logits."""
    f32 = torch.float32
    n, lp, ls = _row_args(logits, None, shape.vocab, shape.dtype, "logits")
    _, dp, ds = _row_args(d_logits, n, shape.vocab, shape.dtype, "d_logits")
    _lib.check(_lib.load().gdn_stack_logprobs_bwd(
        shape._ref, n, lp, ls, _whole(targets, (n,), torch.int32, "targets"), _whole(scale, (n,), f32, "scale"),
        _whole(stats, (n, 2), f32, "stats"), _whole(entropy, (n,), f32, "entropy"),
        _whole(d_logprobs, (n,), f32, "d_logprobs"), _whole(d_entropy, (n,), f32, "d_entropy"), dp, ds,
        _stream(stream, logits, targets, scale, stats, entropy, d_logprobs, d_entropy, d_logits)))


def gdn_stack_distill(shape: LogitsShape, logits, teacher_ids, teacher_values, loss, stats, workspace, scale=None,
                      stream=None) -> None:
    """Divergence of every row's distribution from the teacher's entries, sum p (log p - log q)."""
    f32, k = torch.float32, shape.top
    n, lp, ls = _row_args(logits, None, shape.vocab, shape.dtype, "logits")
    _lib.check(_lib.load().gdn_stack_distill(
        shape._ref, n, lp, ls, _whole(teacher_ids, (n, k), torch.int32, "teacher_ids"),
        _whole(teacher_values, (n, k), f32, "teacher_values"), _whole(scale, (n,), f32, "scale"),
        _whole(loss, (n,), f32, "loss"), _whole(stats, (n, 4), f32, "stats"), *_bytes(workspace),
        _stream(stream, logits, teacher_ids, teacher_values, scale, loss, stats, workspace)))


def gdn_stack_distill_bwd(shape: LogitsShape, logits, teacher_ids, teacher_values, stats, d_loss, d_logits, scale=None,
                          stream=None) -> None:
    """Gradient of the divergence.  d_logits may be logits."""
    f32, k = torch.float32, shape.top
    n, lp, ls = _row_args(logits, None, shape.vocab, shape.dtype, "logits")
    _, dp, ds = _row_args(d_logits, n, shape.vocab, shape.dtype, "d_logits")
    _lib.check(_lib.load().gdn_stack_distill_bwd(
        shape._ref, n, lp, ls, _whole(teacher_ids, (n, k), torch.int32, "teacher_ids"),
        _whole(teacher_values, (n, k), f32, "teacher_values"), _whole(scale, (n,), f32, "scale"),
        _whole(stats, (n, 4), f32, "stats"), _whole(d_loss, (n,), f32, "d_loss"), dp, ds,
        _stream(stream, logits, teacher_ids, teacher_values, scale, stats, d_loss, d_logits)))
