"""Python binding of the 8-bit rows in ``include/rows8.h``.

Argument marshalling only: quantization and restoring run in the library's CUDA
kernels.  ``rows8_quantize`` and ``rows8_restore`` carry the C names and write
into the caller's tensors; ``quantize_rows`` and ``restore_rows`` allocate.
"""

from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib
from ._lib import HESS_BF16, HESS_F16, HESS_F32, check

__all__ = ["Rows8", "rows8_quantize", "rows8_restore", "quantize_rows", "restore_rows"]

_DTYPES = {torch.bfloat16: HESS_BF16, torch.float16: HESS_F16, torch.float32: HESS_F32}


class Rows8(NamedTuple):
    """A [..., d] matrix as int8 ``codes`` [..., d] with fp32 ``scale``s: [...] (or [..., 1]) for group 0,
    one per row; [..., ceil(d / group)] for one per ``group`` columns of a row.  It stands for
    ``codes * scale``."""
    codes: torch.Tensor
    scale: torch.Tensor
    group: int = 0


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
            t.record_stream(stream)


def _written(*tensors) -> None:
    """Autograd learns that a caller's tensors were written, as after an in-place operation."""
    torch.autograd.graph.increment_version(tensors)


def _rows2d(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    """(rows, d, row stride in elements) of a [..., d] tensor whose rows are
    evenly spaced and contiguous inside."""
    shape = t.shape
    if len(shape) == 2 and t.is_cuda and t.is_contiguous() and shape[1]:
        return shape[0], shape[1], shape[1]
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not shape or shape[-1] == 0:
        raise ValueError(f"{name} must have at least one column")
    d = shape[-1]
    if t.is_contiguous():
        return t.numel() // d, d, d
    if len(shape) != 2 or (d > 1 and t.stride(1) != 1) or (shape[0] > 1 and t.stride(0) < d):
        raise ValueError(f"{name} must be contiguous, or a 2-D view whose rows are contiguous")
    return shape[0], d, t.stride(0) if shape[0] > 1 else d


def _float_rows(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return _rows2d(t, name)


def _code_rows(t: torch.Tensor, name: str) -> Tuple[int, int, int]:
    if t.dtype is not torch.int8:
        raise ValueError(f"{name} must be int8, got {t.dtype}")
    return _rows2d(t, name)


def _is_rows(rows, name: str) -> None:
    if not hasattr(rows, "codes"):
        raise ValueError(f"{name} must be 8-bit rows (Rows8), got {type(rows).__name__}")


def _groups(d: int, group: int) -> int:
    return -(-d // group) if group > 0 else 1


def _scale(t: torch.Tensor, n: int, d: int, group: int, name: str) -> int:
    if t.dtype is not torch.float32 or not t.is_cuda or not t.is_contiguous() or \
            t.numel() != (n * _groups(d, group) if group else n):
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of {n} x {_groups(d, group)} scales")
    return t.data_ptr()


def _same_device(first: torch.Tensor, *others: torch.Tensor) -> int:
    dev = first.get_device()
    for t in others:
        if t.get_device() != dev:
            raise ValueError("the tensors are on different devices")
    return dev


def _on(dev: int, call, args) -> None:
    """The call with the tensors' device current."""
    if torch._C._cuda_getDevice() == dev:
        st = call(*args)
    else:
        with torch.cuda.device(dev):
            st = call(*args)
    if st:
        check(st)


def _quantize(X, group, codes, scale, stream) -> None:
    n, d, ldx = _float_rows(X, "X")
    n2, d2, ldc = _code_rows(codes, "codes")
    if (n2, d2) != (n, d):
        raise ValueError(f"codes must be {n} rows of {d}")
    dev = _same_device(X, codes, scale)
    _on(dev, _lib.load().rows8_quantize,
        (X.data_ptr(), ldx, n, d, _DTYPES[X.dtype], int(group), codes.data_ptr(), ldc,
         _scale(scale, n, d, group, "scale"), _stream(stream, dev)))


def rows8_quantize(X: torch.Tensor, group: int, codes_out: torch.Tensor, scale_out: torch.Tensor, stream=None) -> None:
    """Codes and scales of X into the caller's tensors."""
    _quantize(X, group, codes_out, scale_out, stream)
    _written(codes_out, scale_out)
    _used_on(stream, X, codes_out, scale_out)


def _restore(rows: Rows8, X, stream) -> None:
    _is_rows(rows, "rows")
    n, d, ldc = _code_rows(rows.codes, "codes")
    n2, d2, ldx = _float_rows(X, "X_out")
    if (n2, d2) != (n, d):
        raise ValueError(f"X_out must be {n} rows of {d}")
    dev = _same_device(rows.codes, rows.scale, X)
    _on(dev, _lib.load().rows8_restore,
        (rows.codes.data_ptr(), ldc, _scale(rows.scale, n, d, rows.group, "scale"), n, d, int(rows.group),
         X.data_ptr(), ldx, _DTYPES[X.dtype], _stream(stream, dev)))


def rows8_restore(rows: Rows8, X_out: torch.Tensor, stream=None) -> None:
    """The values of ``rows``, rounded once to X_out's type, into the caller's tensor."""
    _restore(rows, X_out, stream)
    _written(X_out)
    _used_on(stream, rows.codes, rows.scale, X_out)


def quantize_rows(X: torch.Tensor, group: int = 0, stream=None) -> Rows8:
    """8-bit rows of X [..., d]: one scale per row (group 0), or per ``group``
    (32, 64, 128 or 256) consecutive columns of a row."""
    n, d, ldx = _float_rows(X, "X")
    shape, device = X.shape, X.device
    wide = (*shape[:-1], _groups(d, group)) if group else shape[:-1]
    if stream is None:
        codes = torch.empty(shape, dtype=torch.int8, device=device)
        scale = torch.empty(wide, dtype=torch.float32, device=device)
    else:
        codes, scale = _empty(shape, torch.int8, X, stream), _empty(wide, torch.float32, X, stream)
        _used_on(stream, X)
    dev = device.index
    _on(dev, _lib.load().rows8_quantize,
        (X.data_ptr(), ldx, n, d, _DTYPES[X.dtype], group, codes.data_ptr(), d, scale.data_ptr(), _stream(stream, dev)))
    return Rows8(codes, scale, group)


def restore_rows(rows: Rows8, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """``codes * scale``, rounded once to ``dtype`` (to ``out``'s type when that is given)."""
    if out is not None:
        rows8_restore(rows, out, stream)
        return out
    if dtype not in _DTYPES:
        raise ValueError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    if isinstance(rows, torch.Tensor):
        _is_rows(rows, "rows")
    codes, scale, group = rows
    n, d, ldc = _code_rows(codes, "codes")
    dev = _same_device(codes, scale)
    from_scale = _scale(scale, n, d, group, "scale")
    if stream is None:
        out = torch.empty(codes.shape, dtype=dtype, device=codes.device)
    else:
        out = _empty(codes.shape, dtype, codes, stream)
        _used_on(stream, codes, scale)
    _on(dev, _lib.load().rows8_restore,
        (codes.data_ptr(), ldc, from_scale, n, d, group, out.data_ptr(), d, _DTYPES[dtype], _stream(stream, dev)))
    return out
