"""Argument checks of the 8-bit calls that need no GPU."""

import ctypes
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()
    from gptq_qqq_calibration_gb300 import _lib
    return _lib.load()


@pytest.mark.parametrize("args,status", [
    ((0, 64, 0, 0, 0), 1), ((64, -8, 0, 0, 0), 1), ((72, 64, 0, 0, 0), 2), ((64, 68, 0, 0, 0), 2),
    ((65552, 64, 0, 0, 0), 2), ((64, 65544, 0, 0, 0), 2), ((64, 64, -1, 0, 0), 1), ((64, 64, 0, -1, 0), 1),
    ((64, 64, (1 << 26) + 1, 0, 0), 2), ((64, 64, 0, (1 << 26) + 1, 0), 2), ((64, 64, 0, 0, 1), 2),
    ((64, 64, 0, 0, 5), 1)])
def test_create_refuses(lib, args, status):
    g = ctypes.c_void_p()
    assert lib.int8_linear_create(*args, ctypes.byref(g)) == status
    assert g.value is None and lib.hess_last_error()
    assert lib.int8_linear_create(*args, None) == 1


def test_null_handles(lib):
    p = ctypes.c_void_p(4096)
    assert lib.int8_linear_forward(None, p, 4, p, p, p, None) == 1
    assert lib.int8_linear_forward_rows8(None, p, p, 4, p, p, p, None) == 1
    assert lib.int8_linear_backward(None, p, 4, p, p, 0, p, p, p, p, None) == 1
    assert lib.int8_linear_sync(None, None) == 1
    assert lib.int8_linear_set_timeout(None, 5) == 1
    assert lib.int8_linear_destroy(None) == 0
    assert lib.gated_ff_reserve_rows8(None) == 1
    assert lib.gated_ff_backward_rows8(None, p, p, 0, 4, p, p, p, p, p, p, None) == 1


@pytest.mark.parametrize("n,d,ldx,ldc,dtype,group,status", [
    (-1, 8, 8, 8, 0, 0, 1), (4, 0, 8, 8, 0, 0, 1), (4, 8, 7, 8, 0, 0, 1), (4, 8, 8, 7, 0, 0, 1), (4, 8, 8, 8, 3, 0, 1),
    (4, 8, 8, 8, 0, -32, 1), (4, 8, 8, 8, 0, 16, 2), (4, 8, 8, 8, 0, 512, 2), (1 << 31, 8, 8, 8, 0, 0, 2),
    (4, (1 << 24) + 1, 1 << 25, 1 << 25, 0, 0, 2), (4, 8, (1 << 28) + 1, 8, 0, 0, 2),
    ((1 << 31) - 1, 1 << 24, 1 << 24, 1 << 24, 0, 0, 2)])
def test_rows8_refuses_sizes(lib, n, d, ldx, ldc, dtype, group, status):
    p = ctypes.c_void_p(4096)
    assert lib.rows8_quantize(p, ldx, n, d, dtype, group, p, ldc, p, None) == status
    assert lib.rows8_restore(p, ldc, p, n, d, group, p, ldx, dtype, None) == status
    assert lib.hess_last_error()


def test_no_rows_is_a_no_op(lib):
    assert lib.rows8_quantize(None, 8, 0, 8, 0, 0, None, 8, None, None) == 0
    assert lib.rows8_restore(None, 8, None, 0, 8, 0, None, 8, 0, None) == 0


def test_injected_allocation_failure_reports_oom():
    code = (
        "import ctypes, sys; sys.path.insert(0, %r)\n"
        "from gptq_qqq_calibration_gb300 import _lib\n"
        "L = _lib.load(); h = ctypes.c_void_p()\n"
        "assert L.int8_linear_create(256, 512, 16, 0, 0, ctypes.byref(h)) == _lib.HESS_ERR_OOM\n"
        "assert h.value is None\n"
        "print('ok')\n" % ROOT)
    env = dict(os.environ, HESS_FAULT="alloc")
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr
