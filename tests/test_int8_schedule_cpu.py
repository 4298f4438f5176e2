"""CPU check of the schedule of the 8-bit integer product on SM pairs.

`int8_schedule_check.cu` is compiled with nvcc as host code. It runs the functions
the kernel and the host library use (`csrc/int8_schedule.cuh`) for some twenty
thousand sizes. It also holds the sizes of the GPU test of split tiles to being
laid out as that test says. A planted mistake in a copy of the schedule must make
it fail.
"""

import os

import pytest

from test_ff_schedule_cpu import run
from test_gpu_int8_linear import LAYOUTS
from test_schedule_cpu import CSRC, ROOT, _nvcc

HEADER = os.path.join(CSRC, "int8_schedule.cuh")
SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "int8_schedule_check.cu")


def build(tmp_path, text=None):
    (tmp_path / "int8_schedule.cuh").write_text(open(HEADER).read() if text is None else text)
    exe = str(tmp_path / "int8_schedule_check")
    rc, out = run(_nvcc(), "-std=c++17", "-O1", "-I", str(tmp_path), "-I", os.path.join(ROOT, "include"), SRC, "-o",
                  exe)
    assert rc == 0, out
    return exe


def test_every_stage_of_every_tile_once(tmp_path):
    exe = build(tmp_path)
    rc, out = run(exe)
    assert rc == 0 and out.startswith("schedule ok"), out
    rc, out = run(exe, *(str(v) for s in LAYOUTS for v in s))
    assert rc == 0, out
    for size, line in zip(LAYOUTS, out.splitlines()):
        tok, rows, whole, parts = map(int, line.split())
        what = LAYOUTS[size]
        assert ("split" in what) == (parts > 1) and ("whole" in what) == (parts > 1 and whole > 0), (size, line)
        assert ("rows" in what) == (rows < 128) and ("tokens" in what) == (size[0] > tok), (size, line)


@pytest.mark.parametrize("old,new", [
    # the pieces of a split tile counted from the wrong tile
    ("r.split = (u - p.whole) / p.parts;", "r.split = u / p.parts;"),
    # a stage left out between two pieces
    ("r.kb0 = n_kb * r.part / r.parts;", "r.kb0 = (n_kb * r.part + r.parts - 1) / r.parts;"),
    # the last group of row tiles taken for a full one
    ("p.tiles_f - g * kGroupF < kGroupF ? p.tiles_f - g * kGroupF : kGroupF", "kGroupF"),
    # more pieces than the workspace holds
    ("(s == 1 || rest * s <= pairs)", "true"),
])
def test_planted_mistakes_fail(tmp_path, old, new):
    text = open(HEADER).read()
    assert text.count(old) == 1, old
    rc, out = run(build(tmp_path, text.replace(old, new)))
    assert rc != 0, out
