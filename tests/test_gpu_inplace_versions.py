"""Results written into a caller's tensor count as an in-place change of it:
an autograd graph that saved the tensor raises in its backward, as it does after
torch's own in-place operations, and does not go on with the new values."""

import pytest
import torch

from test_gpu_distill import make as make_rows
from test_gpu_gated_ff import make as make_ff

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def rows():
    s, v, i, _ = make_rows(5, 300, 6, torch.float32, 3)
    return s.cuda(), v.cuda(), i.cuda()


def test_distill_step_over_logits_that_a_graph_saved():
    from gptq_qqq_calibration_gb300 import distill_loss, distill_step
    S, V, I = rows()
    x = S.clone().requires_grad_()
    logits = torch.tanh(x / 30.0) * 30.0
    loss = distill_loss(logits, V, I)
    distill_step(logits.detach(), V, I, out=logits.detach())
    with pytest.raises(RuntimeError, match="inplace operation"):
        loss.sum().backward()


def test_distill_backward_into_a_tensor_that_a_graph_saved():
    from gptq_qqq_calibration_gb300 import distill_backward, distill_forward
    S, V, I = rows()
    w = torch.randn(5, 300, device="cuda", requires_grad=True)
    out = torch.ones_like(S)
    y = (w * out).sum()  # saves out
    _, stats = distill_forward(S, V, I)
    before = out._version
    distill_backward(S, stats, V, I, out=out)
    assert out._version > before
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.backward()


def test_gated_ff_into_a_tensor_that_a_graph_saved():
    from gptq_qqq_calibration_gb300 import GatedFF
    x, wg, wu, _ = (t.cuda() for t in make_ff(20, 64, 128, torch.bfloat16, 4))
    op = GatedFF(64, 128)
    w = torch.randn(20, 128, device="cuda", requires_grad=True)
    out = torch.ones(20, 128, dtype=torch.bfloat16, device="cuda")
    y = (w * out).sum()
    op.forward(x, wg, wu, out=out)
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.backward()


def test_handle_functions_count_too():
    from gptq_qqq_calibration_gb300.gated_ff import GatedFF, gated_ff_backward, gated_ff_forward
    x, wg, wu, dh = (t.cuda() for t in make_ff(20, 64, 128, torch.bfloat16, 5))
    op = GatedFF(64, 128, train_tokens=20)
    outs = [torch.empty_like(t) for t in (dh, x, wg, wu)]
    before = [t._version for t in outs]
    gated_ff_forward(op.handle, x, 20, wg, wu, outs[0])
    gated_ff_backward(op.handle, x, 20, wg, wu, dh, *outs[1:])
    assert all(t._version > b for t, b in zip(outs, before))
    gated_ff_backward(op.handle, x, 20, wg, wu, dh, None, None, None)
    op.sync()


def test_a_step_over_logits_that_nothing_saved_still_works():
    from gptq_qqq_calibration_gb300 import distill_step
    S, V, I = rows()
    want = distill_step(S, V, I)
    with torch.inference_mode():
        T = S.clone()
        got = distill_step(T, V, I, out=T)
    assert got[1] is T and torch.equal(T, want[1]) and torch.equal(got[0], want[0])
