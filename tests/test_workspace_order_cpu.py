"""CPU check of the order in which calls use a handle's workspace.

`workspace_order_check.cpp` links `csrc/workspace_order.h` against a model of the
CUDA runtime's streams, events and captures and runs random programs on it. It
runs here, without a GPU. A planted mistake in a copy of the header must make it
fail.
"""

import os
import shutil
import subprocess

import pytest

from test_schedule_cpu import _nvcc

HERE = os.path.dirname(os.path.abspath(__file__))
HEADER = os.path.join(os.path.dirname(HERE), "gptq_qqq_calibration_gb300", "csrc", "workspace_order.h")


def run(tmp_path, header, *args):
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    exe = str(tmp_path / "workspace_order_check")
    shutil.copy(header, tmp_path / "workspace_order.h") if os.path.dirname(header) != str(tmp_path) else None
    cmd = ["g++", "-std=c++17", "-O1", "-I", str(tmp_path), "-I", include,
           os.path.join(HERE, "workspace_order_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=300)
    assert r.returncode == 0, r.stdout.decode(errors="replace")
    r = subprocess.run([exe, *args], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=300)
    return r.returncode, r.stdout.decode(errors="replace")


def test_calls_follow_one_another(tmp_path):
    rc, out = run(tmp_path, HEADER)
    assert rc == 0 and out.startswith("order ok"), out


@pytest.mark.parametrize("old,new", [
    # waits inside a capture for work outside it
    ("if (in) return has_capture && capture == id ? cudaStreamWaitEvent(s, captured, 0) : cudaSuccess;\n", ""),
    # the event of the calls outside recorded inside
    ("cudaEventRecord(in ? captured : done, s)", "cudaEventRecord(done, s)"),
    # the calls of an earlier capture waited for
    ("has_capture && capture == id ?", "has_capture ?"),
    # no order within a capture
    ("has_capture && capture == id ? cudaStreamWaitEvent(s, captured, 0) : cudaSuccess", "cudaSuccess"),
])
def test_planted_mistakes_fail(tmp_path, old, new):
    text = open(HEADER).read()
    assert text.count(old) == 1, old
    (tmp_path / "workspace_order.h").write_text(text.replace(old, new))
    rc, out = run(tmp_path, str(tmp_path / "workspace_order.h"))
    assert rc != 0, out
