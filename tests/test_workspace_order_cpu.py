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


def test_equal_handles_may_be_other_streams(tmp_path):
    """Handle values that stand for one stream and later for another: a thread's
    own default stream, or a new stream at a destroyed one's value."""
    rc, out = run(tmp_path, HEADER, "aliases")
    assert rc == 0 and out.startswith("order ok"), out


def planted(tmp_path, old, new, *args):
    text = open(HEADER).read()
    assert text.count(old) == 1, old
    (tmp_path / "workspace_order.h").write_text(text.replace(old, new))
    rc, out = run(tmp_path, str(tmp_path / "workspace_order.h"), *args)
    assert rc != 0, out


@pytest.mark.parametrize("old,new", [
    # waits inside a capture for work outside it, and outside for a capture's
    ("const User& u = in ? inside : outside;", "const User& u = outside;"),
    # an id asked for inside a capture
    ("if (in || s ==", "if (s =="),
    # the event of the calls outside recorded inside
    ("cudaEventRecord(u.event, s)", "cudaEventRecord(outside.event, s)"),
    # the calls of an earlier capture waited for
    ("!u.some || u.capture != now.capture", "!u.some"),
    # no order within a capture
    ("!u.some || u.capture != now.capture", "!u.some || in"),
    # no order outside
    ("!u.some || u.capture != now.capture", "!u.some || u.capture != now.capture || !in"),
])
def test_planted_mistakes_fail(tmp_path, old, new):
    planted(tmp_path, old, new)


@pytest.mark.parametrize("old,new", [
    ("if (in || s == cudaStreamPerThread)", "if (in)"),
    ("return cudaStreamGetId(s, &now.stream);",
     "return now.stream = reinterpret_cast<unsigned long long>(s), cudaSuccess;"),
])
def test_planted_mistakes_with_handles_fail(tmp_path, old, new):
    planted(tmp_path, old, new, "aliases")
