"""Python binding of the 8-bit integer linear layer in ``include/int8_linear.h``.

Argument marshalling only: quantization, the product and the gradients run in
the library's CUDA kernels.  Functions carry the C names; ``Int8Linear`` wraps a
handle and can be called as a node of an autograd graph.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple, Union

import torch

from . import _lib
from ._lib import HESS_BF16, HESS_F16, HESS_F32, check
from .rows8 import Rows8, _is_rows, _scale, _stream, _used_on, _written, quantize_rows

__all__ = ["int8_linear_create", "int8_linear_forward", "int8_linear_forward_rows8", "int8_linear_backward",
           "int8_linear_sync", "int8_linear_set_timeout", "int8_linear_destroy", "Int8Linear"]

_DTYPES = {torch.bfloat16: HESS_BF16, torch.float16: HESS_F16, torch.float32: HESS_F32}


def _empty(shape, like: torch.Tensor, dtype: torch.dtype, stream) -> torch.Tensor:
    """Allocated on the stream that will write it, so that the caching
    allocator orders the memory's former users before the kernel."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def int8_linear_create(d: int, f: int, tokens: int, train_tokens: int, dtype: int) -> int:
    g = ctypes.c_void_p()
    check(_lib.load().int8_linear_create(int(d), int(f), int(tokens), int(train_tokens), int(dtype), ctypes.byref(g)))
    return g.value


def _forward(g, X, n_tokens, W_codes, W_scale, Y_out, stream) -> None:
    st = _lib.load().int8_linear_forward(g, X.data_ptr(), n_tokens, W_codes.data_ptr(), W_scale.data_ptr(),
                                         Y_out.data_ptr(), _stream(stream, X.get_device()))
    if st:
        check(st)


def int8_linear_forward(g: int, X, n_tokens: int, W_codes, W_scale, Y_out, stream=None) -> None:
    _forward(g, X, n_tokens, W_codes, W_scale, Y_out, stream)
    _written(Y_out)


def _forward_rows8(g, X_codes, X_scale, n_tokens, W_codes, W_scale, Y_out, stream) -> None:
    st = _lib.load().int8_linear_forward_rows8(g, X_codes.data_ptr(), X_scale.data_ptr(), n_tokens,
                                               W_codes.data_ptr(), W_scale.data_ptr(), Y_out.data_ptr(),
                                               _stream(stream, X_codes.get_device()))
    if st:
        check(st)


def int8_linear_forward_rows8(g: int, X_codes, X_scale, n_tokens: int, W_codes, W_scale, Y_out, stream=None) -> None:
    _forward_rows8(g, X_codes, X_scale, n_tokens, W_codes, W_scale, Y_out, stream)
    _written(Y_out)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _backward(g, dY, n_tokens, X_codes, X_scale, group, W_codes, W_scale, dX_out, dW_out, stream) -> None:
    st = _lib.load().int8_linear_backward(g, dY.data_ptr(), n_tokens, _ptr(X_codes), _ptr(X_scale), group,
                                          _ptr(W_codes), _ptr(W_scale), _ptr(dX_out), _ptr(dW_out),
                                          _stream(stream, dY.get_device()))
    if st:
        check(st)


def int8_linear_backward(g: int, dY, n_tokens: int, X_codes, X_scale, group: int, W_codes, W_scale, dX_out, dW_out,
                         stream=None) -> None:
    _backward(g, dY, n_tokens, X_codes, X_scale, group, W_codes, W_scale, dX_out, dW_out, stream)
    _written(*(t for t in (dX_out, dW_out) if t is not None))


def int8_linear_sync(g: int, stream=None) -> None:
    check(_lib.load().int8_linear_sync(g, _stream(stream, torch.cuda.current_device())))


def int8_linear_set_timeout(g: int, ns: int) -> None:
    check(_lib.load().int8_linear_set_timeout(g, int(ns)))


def int8_linear_destroy(g: int) -> None:
    check(_lib.load().int8_linear_destroy(g))


class Int8Linear:
    """``y = (qx qw^T) * sx * sw`` for one pair of widths (d inputs, f outputs).

    Weights are 8-bit rows [f, d] with one scale per output channel
    (``quantize_rows(W)``, or ``Rows8(codes, scales)`` from ``GPTQ.quantize`` with
    group_size -1); they belong to the caller, so one object serves every layer of
    these widths.  Activations come in the object's type and are quantized per token
    on the way, or as 8-bit rows.  ``tokens`` is the most tokens a forward call will
    have, ``train_tokens`` the most of a backward call.

    Called as a function, ``op(X, W)`` with a 16-bit or fp32 master weight, the
    object is a node of an autograd graph: it quantizes both, keeps their 8-bit rows
    for the backward pass, and sends gradients straight through the roundings.  Gradients
    are made in fp32 sums and rounded to the object's type, that of an fp32 master weight too.
    A captured backward pass belongs into the capture of its forward pass, with no
    other graph of the same leaf tensors alive.

    The object's calls may come on any streams, and may be captured into CUDA
    graphs.  Replays of such graphs are the caller's to order, with each other
    and with the object's other calls: they share its workspace, and need the
    object to stay alive.
    """

    def __init__(self, d: int, f: int, tokens: int, train_tokens: int = 0, dtype: torch.dtype = torch.bfloat16):
        self.handle = None
        if dtype not in _DTYPES:
            raise ValueError(f"dtype must be bfloat16 or float16, got {dtype}")
        self.d, self.f, self.dtype = int(d), int(f), dtype
        self.handle = int8_linear_create(d, f, tokens, train_tokens, _DTYPES[dtype])

    def _rows(self, t: torch.Tensor, name: str, width: int, dtype: torch.dtype) -> int:
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
        if not t.dim() or t.shape[-1] != width:
            raise ValueError(f"{name} must have a last dimension of {width}")
        return t.numel() // width

    def _weight(self, weight: Rows8) -> None:
        _is_rows(weight, "weight")
        if weight.group != 0:
            raise ValueError("the weight must have one scale per output channel (group 0)")
        if self._rows(weight.codes, "weight.codes", self.d, torch.int8) != self.f:
            raise ValueError(f"weight.codes must be [{self.f}, {self.d}]")
        _scale(weight.scale, self.f, self.d, 0, "weight.scale")

    def forward(self, X: Union[torch.Tensor, Rows8], weight: Rows8, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """y of X [..., d] (the object's type, or 8-bit rows with group 0); ``out`` shares no
        memory with the inputs."""
        self._weight(weight)
        kept = isinstance(X, Rows8)
        if kept:
            if X.group != 0:
                raise ValueError("X must have one scale per token (group 0)")
            n, like = self._rows(X.codes, "X.codes", self.d, torch.int8), X.codes
            _scale(X.scale, n, self.d, 0, "X.scale")
        else:
            n, like = self._rows(X, "X", self.d, self.dtype), X
        given = out
        if out is None:
            out = _empty((*like.shape[:-1], self.f), like, self.dtype, stream)
        elif self._rows(out, "out", self.f, self.dtype) != n:
            raise ValueError(f"out must have {n} rows")
        if kept:
            _forward_rows8(self.handle, X.codes, X.scale, n, weight.codes, weight.scale, out, stream)
            _used_on(stream, X.codes, X.scale, weight.codes, weight.scale, out)
        else:
            _forward(self.handle, X, n, weight.codes, weight.scale, out, stream)
            _used_on(stream, X, weight.codes, weight.scale, out)
        if given is not None:
            _written(out)
        return out

    def backward(self, dY: torch.Tensor, X: Rows8, weight: Rows8, want_dx: bool = True, want_dw: bool = True,
                 stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
        """(dX, dW) from the 8-bit rows that forward read (or an 8-bit checkpoint of
        them, any group); None for what is not wanted."""
        self._weight(weight)
        _is_rows(X, "X")
        n = self._rows(dY, "dY", self.f, self.dtype)
        if self._rows(X.codes, "X.codes", self.d, torch.int8) != n:
            raise ValueError(f"X must have {n} rows")
        _scale(X.scale, n, self.d, X.group, "X.scale")
        dx = _empty(X.codes.shape, dY, self.dtype, stream) if want_dx else None
        dw = _empty((self.f, self.d), dY, self.dtype, stream) if want_dw else None
        _backward(self.handle, dY, n, X.codes, X.scale, int(X.group), weight.codes, weight.scale, dx, dw, stream)
        _used_on(stream, dY, X.codes, X.scale, weight.codes, weight.scale)
        return dx, dw

    def __call__(self, X: torch.Tensor, W: torch.Tensor) -> torch.Tensor:
        return _Int8Linear.apply(self, X, W)

    def sync(self, stream=None) -> None:
        int8_linear_sync(self.handle, stream)

    def close(self) -> None:
        if self.handle:
            int8_linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _Int8Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, op, X, W):
        rows, weight = quantize_rows(X), quantize_rows(W)
        ctx.op = op
        ctx.save_for_backward(*rows[:2], *weight[:2])
        return op.forward(rows, weight)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dY):
        x_codes, x_scale, w_codes, w_scale = ctx.saved_tensors
        want = ctx.needs_input_grad
        dY = dY.contiguous()
        if dY.data_ptr() % 16:  # a part of a buffer that starts anywhere
            dY = dY.clone()
        dx, dw = ctx.op.backward(dY, Rows8(x_codes, x_scale), Rows8(w_codes, w_scale), want_dx=want[1],
                                 want_dw=want[2])
        return None, dx, dw
