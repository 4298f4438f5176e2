"""Feed-forward calls whose tiles are split along their sums, against float64.

A test that needs no GPU (test_ff_schedule_cpu.py) holds the sizes to being
split as they are listed here.  Bounds: those of test_gpu_gated_ff.py, whose sums
of K products also cover the pieces, added in fp32."""

import pytest
import torch

from test_gpu_gated_ff import check, make, reference

pytestmark = pytest.mark.gpu

# tokens, d, f: (whole tiles, units of each tile after them, units of a tile of dX) with 76 pairs
SPLIT = {
    (300, 2568, 1096): (0, 3, 1),
    (129, 4104, 264): (0, 4, 1),
    (140, 8192, 136): (0, 5, 1),
    (2100, 2568, 1096): (76, 3, 1),
    (600, 2568, 3208): (76, 3, 1),
    (140, 264, 5000): (40, 1, 6),
    (513, 1032, 2504): (60, 1, 3),
}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


@pytest.mark.parametrize("dtype,kind", [(torch.bfloat16, "silu"), (torch.float16, "gelu_tanh")])
@pytest.mark.parametrize("n,d,f", list(SPLIT))
def test_split_tiles(n, d, f, dtype, kind):
    from gptq_qqq_calibration_gb300 import GatedFF
    data = make(n, d, f, dtype, n + d)
    ref = reference(*data, kind)
    op = GatedFF(d, f, train_tokens=n, dtype=dtype, activation=kind)
    args = [t.cuda() for t in data]
    first = (op.forward(*args[:3]), *op.backward(*args))
    for got, k in zip(first, ("h", "dx", "dwg", "dwu")):
        check(got, ref[k], dtype)
    # the same bits each time, with whatever the calls before left in the workspace
    other = [t.cuda() for t in make(n, d, f, dtype, n + d + 1)]
    op.forward(*other[:3]), op.backward(*other)
    again = (op.forward(*args[:3]), *op.backward(*args))
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    op.sync()


@pytest.mark.parametrize("n,d,f", [(300, 2568, 1096), (2100, 2568, 1096)])
def test_split_calls_of_several_streams(n, d, f):
    from gptq_qqq_calibration_gb300 import GatedFF
    sets = [[t.cuda() for t in make(n, d, f, torch.bfloat16, 5 + k)] for k in range(3)]
    op = GatedFF(d, f, train_tokens=n)
    want = [(op.forward(*s[:3]), *op.backward(*s)) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        got = [(op.forward(*s[:3], stream=st), *op.backward(*s, stream=st)) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    op.sync()
