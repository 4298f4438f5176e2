"""Gradients that reach the feed-forward node in forms that its kernels do not
take as they come."""

import pytest
import torch

from test_gpu_gated_ff import check, make, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


@pytest.mark.parametrize("before", [1, 3, 8])
def test_gradient_at_an_odd_place_of_a_buffer(before):
    """The gradient of a concatenation's part is a contiguous view that starts
    where the part starts, on any element: the node takes it all the same."""
    from gptq_qqq_calibration_gb300 import GatedFF
    n, d, f = 24, 64, 88
    x, wg, wu, dh = make(n, d, f, torch.bfloat16, 8)
    ref = reference(x, wg, wu, dh, "silu")
    op = GatedFF(d, f, train_tokens=n)
    X, G, U = (t.cuda().requires_grad_() for t in (x, wg, wu))
    joined = torch.cat([torch.zeros(before, dtype=torch.bfloat16, device="cuda"), op(X, G, U).flatten()])
    joined.backward(torch.cat([torch.zeros(before, dtype=torch.bfloat16), dh.flatten()]).cuda())
    for t, k in ((X, "dx"), (G, "dwg"), (U, "dwu")):
        check(t.grad, ref[k], torch.bfloat16)
    op.sync()
