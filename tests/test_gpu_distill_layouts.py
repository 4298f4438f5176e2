"""Distillation rows whose logits and gradients lie between each other in one buffer."""

import pytest
import torch

from test_gpu_distill import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,vocab,gap,first", [(5, 1237, 0, True), (7, 1237, 3, False), (3, 40001, 0, True),
                                                  (64, 5000, 8, False)])
def test_columns_of_one_buffer(rows, vocab, gap, first, dtype):
    from gptq_qqq_calibration_gb300 import distill_backward, distill_forward, distill_step
    s, v, i, t = make(rows, vocab, 9, dtype, vocab + rows)
    kw = dict(top_logits=v.cuda(), top_index=i.cuda(), teacher_lse=torch.logsumexp(t, 1).float().cuda())
    buf = torch.full((rows, 2 * vocab + gap), 7.0, dtype=dtype, device="cuda")
    left, right = buf[:, :vocab], buf[:, vocab + gap:]
    S, out = (left, right) if first else (right, left)
    S.copy_(s)
    # the same rows (their bits depend on where they start in 16 bytes), results elsewhere
    want = distill_step(S, **kw)
    loss, stats = distill_forward(S, **kw)
    want_backward = distill_backward(S, stats, **kw)
    check(s, v, i, want[0].cpu(), want[1].cpu(), 1.0, kw["teacher_lse"].cpu())
    got = distill_step(S, out=out, **kw)
    assert got[1] is out and torch.equal(got[0], want[0]) and torch.equal(out, want[1]) and torch.equal(S, s.cuda())
    assert (buf[:, vocab:vocab + gap] == 7).all()
    out.fill_(3.0)
    distill_backward(S, stats, out=out, **kw)
    assert torch.equal(out, want_backward) and torch.equal(S, s.cuda())
    assert (buf[:, vocab:vocab + gap] == 7).all()
