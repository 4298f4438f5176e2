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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mask", ["-inf", "lowest"])
def test_everything_outside_the_list_masked(dtype, mask):
    """The teacher has a mass where the student has none: an infinite loss, no
    gradient outside the list, q - p inside it."""
    from gptq_qqq_calibration_gb300 import distill_backward, distill_forward, distill_step
    s, v, i, t = make(3, 3000, 10, dtype, 5)
    low = -float("inf") if mask == "-inf" else torch.finfo(dtype).min
    keep = torch.zeros(3, 3000, dtype=torch.bool)
    keep.scatter_(1, i.long(), True)
    s[:2] = torch.where(keep[:2], s[:2], torch.tensor(low, dtype=dtype))
    lse = torch.logsumexp(t, 1).float() + 0.2
    kw = dict(top_logits=v.cuda(), top_index=i.cuda(), teacher_lse=lse.cuda())
    loss, d = distill_step(s.cuda(), **kw)
    loss2, stats = distill_forward(s.cuda(), **kw)
    d2 = distill_backward(s.cuda(), stats, **kw)
    assert torch.isinf(loss[:2]).all() and (loss[:2] > 0).all() and torch.equal(loss, loss2)
    for g in (d.cpu(), d2.cpu()):
        assert not g[:2][~keep[:2]].any()
        check(s[2:], v[2:], i[2:], loss.cpu()[2:], g[2:], 1.0, lse[2:])
        check(torch.where(keep, s, torch.tensor(-float("inf"), dtype=dtype))[:2], v[:2], i[:2], None, g[:2], 1.0,
              lse[:2])


def test_nan_of_the_teacher():
    from gptq_qqq_calibration_gb300 import distill_step
    s, v, i, t = make(3, 500, 6, torch.float32, 6)
    lse = torch.logsumexp(t, 1).float()
    v[0, 2] = float("nan")
    for l in (None, lse.clone()):
        if l is not None:
            l[1] = float("nan")
        loss, d = distill_step(s.cuda(), v.cuda(), i.cuda(), teacher_lse=None if l is None else l.cuda())
        bad = [0] if l is None else [0, 1]
        for r in range(3):
            assert bool(torch.isnan(loss[r])) == (r in bad)
        assert torch.isnan(d[0, i[0, 2].long()])
        if l is not None:
            assert torch.isnan(d[1, i[1].long().cuda()]).all()
        check(s[2:], v[2:], i[2:], loss.cpu()[2:], d.cpu()[2:], 1.0, None if l is None else l[2:])
