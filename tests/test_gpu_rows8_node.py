"""What the feed-forward node of an object with 8-bit checkpoints keeps, and when."""

import pytest
import torch

from test_gpu_gated_ff import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def test_node_keeps_nothing_where_no_input_has_a_gradient(monkeypatch):
    from gptq_qqq_calibration_gb300 import GatedFF, gated_ff
    n, d, f = 48, 256, 384
    x, wg, wu, dh = (t.cuda() for t in make(n, d, f, torch.bfloat16, 4))
    op = GatedFF(d, f, train_tokens=n, rows8=True)
    kept, quantize = [], gated_ff.quantize_rows
    monkeypatch.setattr(gated_ff, "quantize_rows", lambda *a, **k: (kept.append(1), quantize(*a, **k))[1])
    h = op(x, wg, wu)
    assert not h.requires_grad and not kept and torch.equal(h, op.forward(x, wg, wu))
    for which in range(3):
        t = [v.clone() for v in (x, wg, wu)]
        t[which].requires_grad_()
        op(*t).backward(dh)
        assert len(kept) == which + 1
        assert [v.grad is not None for v in t] == [k == which for k in range(3)]
    op.sync()
