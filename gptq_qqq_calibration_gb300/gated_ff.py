"""Python binding of the gated feed-forward projections in ``include/gated_ff.h``.

Argument marshalling only: the projections, the activation and the gradients
run in the library's CUDA kernels.  Functions carry the C names; ``GatedFF``
wraps a handle and can be called as a node of an autograd graph.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple, Union

import torch

from . import _lib
from ._lib import HESS_BF16, HESS_F16, HESS_F32, check
from .rows8 import Rows8, _scale, quantize_rows

__all__ = ["gated_ff_create", "gated_ff_forward", "gated_ff_backward", "gated_ff_reserve_rows8",
           "gated_ff_backward_rows8", "gated_ff_sync", "gated_ff_set_timeout", "gated_ff_destroy", "GatedFF"]

_DTYPES = {torch.bfloat16: HESS_BF16, torch.float16: HESS_F16, torch.float32: HESS_F32}
ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}


def _stream(stream, device: int) -> int:
    if stream is not None:
        return stream.cuda_stream
    # the raw handle of the device's current stream, without building a Stream object
    return torch._C._cuda_getCurrentRawStream(device)


def _empty(shape, like: torch.Tensor, stream) -> torch.Tensor:
    """Allocated on the stream that will write it, so that the caching
    allocator orders the memory's former users before the kernel."""
    if stream is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=like.dtype, device=like.device)


def _used_on(stream, *tensors) -> None:
    """Tensors of another stream stay allocated until `stream` is done with them."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def gated_ff_create(d: int, f: int, train_tokens: int, dtype: int, act: int) -> int:
    g = ctypes.c_void_p()
    check(_lib.load().gated_ff_create(int(d), int(f), int(train_tokens), int(dtype), int(act), ctypes.byref(g)))
    return g.value


def _written(*tensors) -> None:
    """Autograd learns that a caller's tensors were written, as after an in-place operation."""
    torch.autograd.graph.increment_version([t for t in tensors if t is not None])


def _forward(g: int, X, n_tokens: int, W_gate, W_up, H_out, stream) -> None:
    st = _lib.load().gated_ff_forward(g, X.data_ptr(), n_tokens, W_gate.data_ptr(), W_up.data_ptr(),
                                      H_out.data_ptr(), _stream(stream, X.get_device()))
    if st:
        check(st)


def gated_ff_forward(g: int, X, n_tokens: int, W_gate, W_up, H_out, stream=None) -> None:
    _forward(g, X, n_tokens, W_gate, W_up, H_out, stream)
    _written(H_out)


def _backward(g: int, X, n_tokens: int, W_gate, W_up, dH, dX_out, dW_gate_out, dW_up_out, stream) -> None:
    st = _lib.load().gated_ff_backward(
        g, X.data_ptr(), n_tokens, W_gate.data_ptr(), W_up.data_ptr(), dH.data_ptr(),
        None if dX_out is None else dX_out.data_ptr(), None if dW_gate_out is None else dW_gate_out.data_ptr(),
        None if dW_up_out is None else dW_up_out.data_ptr(), _stream(stream, X.get_device()))
    if st:
        check(st)


def gated_ff_backward(g: int, X, n_tokens: int, W_gate, W_up, dH, dX_out, dW_gate_out, dW_up_out,
                      stream=None) -> None:
    _backward(g, X, n_tokens, W_gate, W_up, dH, dX_out, dW_gate_out, dW_up_out, stream)
    _written(dX_out, dW_gate_out, dW_up_out)


def gated_ff_reserve_rows8(g: int) -> None:
    check(_lib.load().gated_ff_reserve_rows8(g))


def _backward_rows8(g: int, X_codes, X_scale, group, n_tokens, W_gate, W_up, dH, dX_out, dW_gate_out, dW_up_out,
                    stream) -> None:
    st = _lib.load().gated_ff_backward_rows8(
        g, X_codes.data_ptr(), X_scale.data_ptr(), group, n_tokens, W_gate.data_ptr(), W_up.data_ptr(), dH.data_ptr(),
        None if dX_out is None else dX_out.data_ptr(), None if dW_gate_out is None else dW_gate_out.data_ptr(),
        None if dW_up_out is None else dW_up_out.data_ptr(), _stream(stream, dH.get_device()))
    if st:
        check(st)


def gated_ff_backward_rows8(g: int, X_codes, X_scale, group: int, n_tokens: int, W_gate, W_up, dH, dX_out,
                            dW_gate_out, dW_up_out, stream=None) -> None:
    _backward_rows8(g, X_codes, X_scale, group, n_tokens, W_gate, W_up, dH, dX_out, dW_gate_out, dW_up_out, stream)
    _written(dX_out, dW_gate_out, dW_up_out)


def gated_ff_sync(g: int, stream=None) -> None:
    check(_lib.load().gated_ff_sync(g, _stream(stream, torch.cuda.current_device())))


def gated_ff_set_timeout(g: int, ns: int) -> None:
    check(_lib.load().gated_ff_set_timeout(g, int(ns)))


def gated_ff_destroy(g: int) -> None:
    check(_lib.load().gated_ff_destroy(g))


class GatedFF:
    """``h = act(x W_gate^T) * (x W_up^T)`` for one pair of widths (d, f).

    ``forward`` and ``backward`` take [..., d] and [..., f] tensors of the
    object's type; weights are [f, d] and belong to the caller, so one object
    serves every layer of these widths.  ``train_tokens`` is the most tokens a
    backward call will have (its workspace is 4 f bytes a token); a backward of
    more is refused, a forward is not.  Called as a function, the object is a node
    of an autograd graph.  With ``rows8`` the object can take 8-bit rows in the place of
    X in ``backward`` (2 d bytes of workspace a token of ``train_tokens``), and the node keeps X
    in that form, with a scale per 128 columns: 1.03 bytes a value instead of 2.  A captured
    backward pass belongs into the capture of its forward pass, with no other graph of
    the same leaf tensors alive.

    The object's calls may come on any streams, and may be captured into CUDA
    graphs.  Replays of such graphs are the caller's to order, with each other
    and with the object's other calls: they share its workspace, and need the
    object to stay alive.
    """

    def __init__(self, d: int, f: int, train_tokens: int = 0, dtype: torch.dtype = torch.bfloat16,
                 activation: str = "silu", rows8: bool = False):
        self.handle = None
        if dtype not in _DTYPES:
            raise ValueError(f"dtype must be bfloat16 or float16, got {dtype}")
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
        self.d, self.f, self.dtype = int(d), int(f), dtype
        self.handle = gated_ff_create(d, f, train_tokens, _DTYPES[dtype], ACTIVATIONS[activation])
        self.rows8 = bool(rows8)
        if rows8:
            gated_ff_reserve_rows8(self.handle)

    def _rows(self, t: torch.Tensor, name: str, width: int) -> int:
        if t.dtype is self.dtype and t.is_cuda and t.is_contiguous() and t.dim() and t.shape[-1] == width:
            return t.numel() // width
        if t.dtype is not self.dtype:
            raise ValueError(f"{name} must be {self.dtype}, got {t.dtype}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
        raise ValueError(f"{name} must have a last dimension of {width}")

    def _kept(self, X: Rows8) -> int:
        codes = X.codes
        if codes.dtype is not torch.int8 or not codes.is_cuda or not codes.is_contiguous() or not codes.dim() or \
                codes.shape[-1] != self.d:
            raise ValueError(f"X.codes must be a contiguous int8 CUDA tensor with a last dimension of {self.d}")
        n = codes.numel() // self.d
        _scale(X.scale, n, self.d, X.group, "X.scale")
        return n

    @staticmethod
    def _not_rows(X) -> None:
        if isinstance(X, Rows8):
            raise ValueError("X must be a tensor here: 8-bit rows are taken by backward")

    def _inputs(self, X, W_gate, W_up) -> int:
        n = self._kept(X) if isinstance(X, Rows8) else self._rows(X, "X", self.d)
        if self._rows(W_gate, "W_gate", self.d) != self.f or self._rows(W_up, "W_up", self.d) != self.f:
            raise ValueError(f"W_gate and W_up must be [{self.f}, {self.d}]")
        return n

    def forward(self, X: torch.Tensor, W_gate: torch.Tensor, W_up: torch.Tensor,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """h of X [..., d]; ``out`` shares no memory with the inputs."""
        self._not_rows(X)
        n = self._inputs(X, W_gate, W_up)
        if out is None:
            out = _empty((n, self.f) if X.dim() == 2 else (*X.shape[:-1], self.f), X, stream)
            _forward(self.handle, X, n, W_gate, W_up, out, stream)
        else:
            if self._rows(out, "out", self.f) != n:
                raise ValueError(f"out must have {n} rows")
            gated_ff_forward(self.handle, X, n, W_gate, W_up, out, stream)
        _used_on(stream, X, W_gate, W_up, out)
        return out

    def backward(self, X: Union[torch.Tensor, Rows8], W_gate: torch.Tensor, W_up: torch.Tensor, dH: torch.Tensor,
                 want_dx: bool = True, want_dw: bool = True, stream=None
                 ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor], Optional[torch.Tensor]]:
        """(dX, dW_gate, dW_up); None for what is not wanted.  X may be an 8-bit
        checkpoint of the input (an object with ``rows8``)."""
        n = self._inputs(X, W_gate, W_up)
        kept = isinstance(X, Rows8)
        if self._rows(dH, "dH", self.f) != n:
            raise ValueError(f"dH must have {n} rows")
        dx = _empty(X.codes.shape if kept else X.shape, dH, stream) if want_dx else None
        dwg = _empty(W_gate.shape, dH, stream) if want_dw else None
        dwu = _empty(W_up.shape, dH, stream) if want_dw else None
        if kept:
            _backward_rows8(self.handle, X.codes, X.scale, int(X.group), n, W_gate, W_up, dH, dx, dwg, dwu, stream)
            _used_on(stream, X.codes, X.scale, W_gate, W_up, dH)
        else:
            _backward(self.handle, X, n, W_gate, W_up, dH, dx, dwg, dwu, stream)
            _used_on(stream, X, W_gate, W_up, dH)
        return dx, dwg, dwu

    def __call__(self, X: torch.Tensor, W_gate: torch.Tensor, W_up: torch.Tensor) -> torch.Tensor:
        self._not_rows(X)
        if self.rows8 and not torch.is_grad_enabled():  # nothing to keep
            return self.forward(X, W_gate, W_up)
        return _GatedFF.apply(self, X, W_gate, W_up)

    def sync(self, stream=None) -> None:
        gated_ff_sync(self.handle, stream)

    def close(self) -> None:
        if self.handle:
            gated_ff_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class _GatedFF(torch.autograd.Function):
    @staticmethod
    def forward(ctx, op, X, W_gate, W_up):
        ctx.op = op
        if not any(ctx.needs_input_grad):  # nothing to keep
            return op.forward(X, W_gate, W_up)
        if op.rows8:
            ctx.save_for_backward(*quantize_rows(X, group=128)[:2], W_gate, W_up)
        else:
            ctx.save_for_backward(X, W_gate, W_up)
        return op.forward(X, W_gate, W_up)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dH):
        *X, W_gate, W_up = ctx.saved_tensors
        X = Rows8(*X, 128) if ctx.op.rows8 else X[0]
        want = ctx.needs_input_grad
        dH = dH.contiguous()
        if dH.data_ptr() % 16:  # a part of a buffer that starts anywhere
            dH = dH.clone()
        dx, dwg, dwu = ctx.op.backward(X, W_gate, W_up, dH, want_dx=want[1],
                                       want_dw=want[2] or want[3])
        return None, dx, dwg if want[2] else None, dwu if want[3] else None
