"""Feed-forward calls that are refused on a GPU: outputs in the memory of
inputs or of each other.  Nothing is launched."""

import pytest
import torch

from test_gpu_gated_ff import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


@pytest.mark.parametrize("n", [16, 200])
def test_forward_over_its_inputs(n):
    from gptq_qqq_calibration_gb300 import GatedFF, HessError
    w = 128  # d == f
    x, wg, wu, _ = (t.cuda() for t in make(n, w, w, torch.bfloat16, 1))
    op = GatedFF(w, w)
    want = op.forward(x, wg, wu)
    buf = torch.empty((2 * n, w), dtype=torch.bfloat16, device="cuda")
    buf[:n] = x
    for at in (0, 1, n // 2, n - 1):
        with pytest.raises(HessError, match="overlaps"):
            op.forward(buf[:n], wg, wu, out=buf[at:at + n])
    weights = torch.cat([wg, wu, torch.zeros_like(x)])
    with pytest.raises(HessError, match="overlaps"):
        op.forward(x, weights[:w], weights[w:2 * w], out=weights[2 * w - 1:2 * w - 1 + n])
    assert torch.equal(buf[:n], x) and torch.equal(weights[:2 * w], torch.cat([wg, wu]))
    # right behind its inputs
    op.forward(buf[:n], wg, wu, out=buf[n:])
    op.forward(x, weights[:w], weights[w:2 * w], out=weights[2 * w:])
    assert torch.equal(buf[n:], want) and torch.equal(weights[2 * w:], want)
    op.sync()


def test_backward_over_its_inputs_or_other_outputs():
    from gptq_qqq_calibration_gb300 import GatedFF, HessError
    from gptq_qqq_calibration_gb300.gated_ff import gated_ff_backward
    n, d, f = 64, 128, 256
    x, wg, wu, dh = (t.cuda() for t in make(n, d, f, torch.bfloat16, 2))
    op = GatedFF(d, f, train_tokens=n)
    want = op.backward(x, wg, wu, dh)
    dx, dw = torch.empty_like(x), torch.empty((2 * f, d), dtype=torch.bfloat16, device="cuda")
    for outs in ((x, dw[:f], dw[f:]), (dx, wg, dw[f:]), (dx, dw[:f], wu), (dx, dw[:f], dw[1:f + 1]),
                 (dw[f - 1:f - 1 + n], dw[:f], dw[f:]), (dh.view(-1)[:n * d].view(n, d), None, None)):
        with pytest.raises(HessError, match="overlaps"):
            gated_ff_backward(op.handle, x, n, wg, wu, dh, *outs)
    gated_ff_backward(op.handle, x, n, wg, wu, dh, dx, dw[:f], dw[f:])
    assert torch.equal(dx, want[0]) and torch.equal(dw[:f], want[1]) and torch.equal(dw[f:], want[2])
    op.sync()
