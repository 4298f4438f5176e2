"""CPU check of the schedule of the feed-forward kernels of SM pairs.

`ff_schedule_check.cu` is compiled with nvcc as host code. It runs the functions
the kernels and the host library use (`csrc/gated_ff_schedule.cuh`) for several
thousand sizes. It also holds the sizes of the GPU test of split tiles to being
split. A planted mistake in a copy of the schedule must make it fail.
"""

import os
import subprocess

import pytest

from test_gpu_gated_ff_split import SPLIT
from test_schedule_cpu import CSRC, ROOT, _nvcc

HEADER = os.path.join(CSRC, "gated_ff_schedule.cuh")
SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "ff_schedule_check.cu")


def build(tmp_path, text=None):
    (tmp_path / "gated_ff_schedule.cuh").write_text(open(HEADER).read() if text is None else text)
    exe = str(tmp_path / "ff_schedule_check")
    cmd = [_nvcc(), "-std=c++17", "-O1", "-I", str(tmp_path), "-I", os.path.join(ROOT, "include"), SRC, "-o", exe]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=300)
    assert r.returncode == 0, r.stdout.decode(errors="replace")
    return exe


def run(*cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=300)
    return r.returncode, r.stdout.decode(errors="replace")


def test_every_box_of_every_tile_once(tmp_path):
    exe = build(tmp_path)
    rc, out = run(exe)
    assert rc == 0 and out.startswith("schedule ok"), out
    rc, out = run(exe, *(str(v) for s in SPLIT for v in s))
    assert rc == 0 and [tuple(map(int, line.split())) for line in out.splitlines()] == list(SPLIT.values()), out


@pytest.mark.parametrize("old,new", [
    # the pieces of a split tile counted from the wrong tile
    ("r.split = (u - p.whole) / p.parts;", "r.split = u / p.parts;"),
    # a box left out between two pieces
    ("r.kb0 = n_kb * r.part / r.parts;", "r.kb0 = (n_kb * r.part + r.parts - 1) / r.parts;"),
    # one turn of the tiles of dW given twice
    ("p.skip * (n_pairs - more) + (turn - p.skip) * n_pairs + pair", "p.skip * (n_pairs - more) + (turn - 1) * n_pairs + pair"),
    # tiles split in more pieces than the workspace holds
    ("s <= 8 && tiles * s <= pairs; ++s", "s <= 8; ++s"),
])
def test_planted_mistakes_fail(tmp_path, old, new):
    text = open(HEADER).read()
    assert text.count(old) == 1, old
    rc, out = run(build(tmp_path, text.replace(old, new)))
    assert rc != 0, out
