"""Python binding of the distillation loss in ``include/distill.h``.

Argument marshalling only: tensors become device pointers, sizes and row
strides; the loss and its gradient run in the library's CUDA kernels.  The
functions carry the C names and allocate their outputs; a gradient written
into a caller's tensor (``out``) is an in-place change of it for autograd.
``distill_loss`` is the same loss as a node of an autograd graph.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import HESS_BF16, HESS_F16, HESS_F32, check

__all__ = ["distill_forward", "distill_backward", "distill_step", "distill_loss"]

_DTYPES = {torch.bfloat16: HESS_BF16, torch.float16: HESS_F16, torch.float32: HESS_F32}
_STATS = 8  # floats of one row of the statistics (DISTILL_STATS)


def _stream(stream, device: int) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the raw handle of the device's current stream, without building a Stream object
    return torch._C._cuda_getCurrentRawStream(device)


def _empty(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """Allocated on the stream that will write it, so that the caching
    allocator orders the memory's former users before the kernel."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _used_on(stream, *tensors) -> None:
    """Tensors of another stream stay allocated until `stream` is done with them."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _rows2d(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """(rows, vocab, row stride in elements) of a [..., vocab] tensor whose
    rows are evenly spaced and contiguous inside."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    shape = t.shape
    if not shape or shape[-1] == 0:
        raise ValueError(f"{name} must have at least one column")
    vocab = shape[-1]
    if t.is_contiguous():
        return t.numel() // vocab, vocab, vocab
    if len(shape) != 2 or (vocab > 1 and t.stride(1) != 1) or (shape[0] > 1 and t.stride(0) < vocab):
        raise ValueError(f"{name} must be contiguous, or a 2-D view whose rows are contiguous")
    return shape[0], vocab, t.stride(0) if shape[0] > 1 else vocab


def _vector(t: Optional[torch.Tensor], rows: int, name: str):
    if t is None:
        return None
    if t.dtype is not torch.float32 or not t.is_cuda or not t.is_contiguous() or t.numel() != rows:
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor with one value a row")
    return t.data_ptr()


def _common(logits, top_logits, top_index, temperature, teacher_lse, weights):
    rows, vocab, ld = _rows2d(logits, "logits")
    top_dtype, index_dtype = top_logits.dtype, top_index.dtype
    if top_dtype not in _DTYPES:
        raise ValueError(f"top_logits must be bfloat16, float16 or float32, got {top_dtype}")
    if index_dtype is not torch.int32 and index_dtype is not torch.int64:
        raise ValueError(f"top_index must be int32 or int64, got {index_dtype}")
    if not (top_logits.is_cuda and top_index.is_cuda and top_logits.is_contiguous() and top_index.is_contiguous()):
        raise ValueError("top_logits and top_index must be contiguous CUDA tensors")
    shape = top_logits.shape
    if not shape or top_index.shape != shape or top_logits.numel() != rows * shape[-1]:
        raise ValueError("top_logits and top_index must both be [rows, top]")
    return rows, (logits.data_ptr(), ld, rows, vocab, _DTYPES[logits.dtype], top_logits.data_ptr(),
                  _DTYPES[top_dtype], top_index.data_ptr(), 4 if index_dtype is torch.int32 else 8, shape[-1],
                  _vector(teacher_lse, rows, "teacher_lse"), _vector(weights, rows, "weights"), temperature)


def _written(out: Optional[torch.Tensor]) -> None:
    """Autograd learns that the caller's tensor was written, as after an in-place operation."""
    if out is not None:
        torch.autograd.graph.increment_version(out)


def _output(out: Optional[torch.Tensor], logits: torch.Tensor, stream) -> Tuple[torch.Tensor, int]:
    if out is None:
        out = _empty(logits.shape, logits.dtype, logits, stream)
        if logits.is_contiguous():
            return out, logits.shape[-1]
    elif out.shape != logits.shape or out.dtype != logits.dtype:
        raise ValueError("the gradient must have the logits' shape and type")
    return out, _rows2d(out, "the gradient")[2]


def distill_forward(logits: torch.Tensor, top_logits: torch.Tensor, top_index: torch.Tensor,
                    temperature: float = 1.0, teacher_lse: Optional[torch.Tensor] = None,
                    weights: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Loss of every row [rows] and the statistics ``distill_backward`` takes."""
    rows, args = _common(logits, top_logits, top_index, temperature, teacher_lse, weights)
    loss = _empty(rows, torch.float32, logits, stream)
    stats = _empty((rows, _STATS), torch.float32, logits, stream)
    check(_lib.load().distill_forward(*args, loss.data_ptr(), stats.data_ptr(), _stream(stream, logits.get_device())))
    _used_on(stream, logits, top_logits, top_index, teacher_lse, weights)
    return loss, stats


def distill_backward(logits: torch.Tensor, stats: torch.Tensor, top_logits: torch.Tensor, top_index: torch.Tensor,
                     temperature: float = 1.0, teacher_lse: Optional[torch.Tensor] = None,
                     weights: Optional[torch.Tensor] = None, grad: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of ``(grad * loss).sum()`` (``loss.sum()`` without grad) with
    respect to the logits; ``out`` may be ``logits``."""
    rows, args = _common(logits, top_logits, top_index, temperature, teacher_lse, weights)
    if not stats.is_cuda or stats.dtype != torch.float32 or not stats.is_contiguous() or \
            stats.numel() != rows * _STATS:
        raise ValueError("stats must be the tensor distill_forward returned for these logits")
    given = out
    out, ldd = _output(out, logits, stream)
    check(_lib.load().distill_backward(*args, stats.data_ptr(), _vector(grad, rows, "grad"), out.data_ptr(), ldd,
                                       _stream(stream, logits.get_device())))
    _written(given)
    _used_on(stream, logits, stats, top_logits, top_index, teacher_lse, weights, grad, out)
    return out


def distill_step(logits: torch.Tensor, top_logits: torch.Tensor, top_index: torch.Tensor, temperature: float = 1.0,
                 teacher_lse: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Loss of every row and the gradient of their sum, in one pass over the
    logits; ``out`` may be ``logits``."""
    rows, args = _common(logits, top_logits, top_index, temperature, teacher_lse, weights)
    loss = _empty(rows, torch.float32, logits, stream)
    given = out
    out, ldd = _output(out, logits, stream)
    check(_lib.load().distill_step(*args, loss.data_ptr(), out.data_ptr(), ldd, _stream(stream, logits.get_device())))
    _written(given)
    _used_on(stream, logits, top_logits, top_index, teacher_lse, weights, out)
    return loss, out


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_logits, top_index, temperature, teacher_lse, weights):
        loss, stats = distill_forward(logits, top_logits, top_index, temperature, teacher_lse, weights)
        ctx.save_for_backward(logits, stats, top_logits, top_index, teacher_lse, weights)
        ctx.temperature = temperature
        return loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        logits, stats, top_logits, top_index, teacher_lse, weights = ctx.saved_tensors
        return (distill_backward(logits, stats, top_logits, top_index, ctx.temperature, teacher_lse, weights,
                                 grad=grad.contiguous()), None, None, None, None, None)


def distill_loss(logits: torch.Tensor, top_logits: torch.Tensor, top_index: torch.Tensor, temperature: float = 1.0,
                 teacher_lse: Optional[torch.Tensor] = None, weights: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Loss of every row [rows] as a node of an autograd graph; only the
    logits get a gradient."""
    return _DistillLoss.apply(logits, top_logits, top_index, float(temperature), teacher_lse, weights)
