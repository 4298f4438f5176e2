"""Argument checks of the distillation calls that need no GPU: everything
here is refused before any CUDA call."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()
    from gptq_qqq_calibration_gb300 import _lib
    return _lib.load()


P = ctypes.c_void_p(4096)  # never dereferenced


def fwd(lib, logits=P, ld=100, rows=4, vocab=100, dtype=0, tv=P, tt=1, ti=P, ib=4, top=5, lse=None, w=None, tau=1.0,
        loss=P, stats=P):
    return lib.distill_forward(logits, ld, rows, vocab, dtype, tv, tt, ti, ib, top, lse, w, tau, loss, stats, None)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(vocab=0), dict(dtype=3), dict(dtype=-1), dict(tt=7), dict(ib=2), dict(ld=99), dict(top=0),
    dict(tau=0.0), dict(tau=float("nan")), dict(tau=1e9), dict(logits=None), dict(tv=None), dict(ti=None),
    dict(loss=None), dict(stats=None), dict(logits=ctypes.c_void_p(4097)), dict(ti=ctypes.c_void_p(4098)),
    dict(stats=ctypes.c_void_p(4104)), dict(w=ctypes.c_void_p(4098))])
def test_invalid(lib, kw):
    from gptq_qqq_calibration_gb300._lib import HESS_ERR_INVALID
    assert fwd(lib, **kw) == HESS_ERR_INVALID
    assert lib.hess_last_error()


def test_unsupported_and_no_rows(lib):
    from gptq_qqq_calibration_gb300._lib import HESS_ERR_INVALID, HESS_ERR_UNSUPPORTED, HESS_OK
    assert fwd(lib, top=1025) == HESS_ERR_UNSUPPORTED
    assert fwd(lib, vocab=(1 << 30) + 1, ld=1 << 31) == HESS_ERR_UNSUPPORTED
    assert fwd(lib, rows=(1 << 27) + 1) == HESS_ERR_UNSUPPORTED
    assert fwd(lib, rows=0, logits=None, tv=None, ti=None, loss=None, stats=None) == HESS_OK
    step = lambda d, ldd, rows=4: lib.distill_step(P, 100, rows, 100, 0, P, 1, P, 4, 5, None, None, 1.0, P, d, ldd, None)  # noqa: E731
    assert step(None, 100) == HESS_ERR_INVALID
    assert step(ctypes.c_void_p(1 << 20), 99) == HESS_ERR_INVALID
    assert step(ctypes.c_void_p(4096 + 16), 100) == HESS_ERR_INVALID  # overlaps without being the logits
    assert step(P, 108) == HESS_ERR_INVALID
    assert step(None, 100, rows=0) == HESS_OK


def test_other_calls_refuse_float16(lib):
    """HESS_F16 is a type of the distillation logits, not of activations."""
    from gptq_qqq_calibration_gb300._lib import HESS_ERR_INVALID, HESS_F16
    out = ctypes.c_void_p(16)
    assert lib.local_hess_compute_noalloc(P, 4, 64, 16, HESS_F16, out, None) == HESS_ERR_INVALID


@pytest.mark.parametrize("dtype,size", [(0, 2), (1, 4)])
def test_rows_between_rows_do_not_overlap(lib, dtype, size):
    """Logits and gradient as columns of one buffer: refused exactly where an
    element of one is an element of the other."""
    rows, vocab, ld = 4, 100, 230
    base = 1 << 20

    def overlaps(shift, ldd=ld, rows=rows, ld=ld):
        lib.distill_step(ctypes.c_void_p(base), ld, rows, vocab, dtype, P, 1, P, 4, 5, None, None, 1.0, P,
                         ctypes.c_void_p(base + shift * size), ldd, None)
        return b"overlaps" in lib.hess_last_error()

    logits = {r * ld + j for r in range(rows) for j in range(vocab)}
    for shift in (*range(-300, 301), 4 * ld - 1, 3 * ld + 99, 3 * ld + 100, -3 * ld - 99, -3 * ld - 100, -4 * ld):
        out = {shift + r * ld + j for r in range(rows) for j in range(vocab)}
        assert overlaps(shift) == (bool(logits & out) and shift != 0), shift
    assert overlaps(105, ldd=ld + 1)  # other strides: by their ranges
    assert not overlaps(0, ldd=100, rows=1)  # one row in place, whatever the strides
    assert not overlaps(0) and not overlaps(4 * ld)


def test_vocabulary_limit(lib):
    """One column past the widest row is refused; the widest is not, here."""
    from gptq_qqq_calibration_gb300._lib import HESS_ERR_UNSUPPORTED
    assert fwd(lib, vocab=(1 << 22) + 1, ld=1 << 23) == HESS_ERR_UNSUPPORTED
    assert b"vocab" in lib.hess_last_error()
    fwd(lib, vocab=1 << 22, ld=1 << 22)
    assert b"vocab" not in lib.hess_last_error()
