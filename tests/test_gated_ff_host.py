"""Argument checks of the gated feed-forward calls that need no GPU."""

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
    ((0, 64, 0, 0, 0), 1), ((64, -8, 0, 0, 0), 1), ((60, 64, 0, 0, 0), 2), ((64, 68, 0, 0, 0), 2),
    ((65544, 64, 0, 0, 0), 2), ((64, 65544, 0, 0, 0), 2), ((64, 64, -1, 0, 0), 1), ((64, 64, (1 << 26) + 1, 0, 0), 2),
    ((64, 64, 0, 1, 0), 2), ((64, 64, 0, 5, 0), 1), ((64, 64, 0, 0, 2), 1)])
def test_create_refuses(lib, args, status):
    g = ctypes.c_void_p()
    assert lib.gated_ff_create(*args, ctypes.byref(g)) == status
    assert g.value is None and lib.hess_last_error()
    assert lib.gated_ff_create(*args, None) == 1


def test_null_handles(lib):
    p = ctypes.c_void_p(4096)
    assert lib.gated_ff_forward(None, p, 4, p, p, p, None) == 1
    assert lib.gated_ff_backward(None, p, 4, p, p, p, p, p, p, None) == 1
    assert lib.gated_ff_sync(None, None) == 1
    assert lib.gated_ff_set_timeout(None, 5) == 1
    assert lib.gated_ff_destroy(None) == 0


def test_injected_allocation_failure_reports_oom():
    code = (
        "import ctypes, sys; sys.path.insert(0, %r)\n"
        "from gptq_qqq_calibration_gb300 import _lib\n"
        "L = _lib.load(); h = ctypes.c_void_p()\n"
        "assert L.gated_ff_create(256, 512, 16, 0, 0, ctypes.byref(h)) == _lib.HESS_ERR_OOM\n"
        "assert h.value is None\n"
        "print('ok')\n" % ROOT)
    env = dict(os.environ, HESS_FAULT="alloc")
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "ok" in r.stdout, r.stderr
