"""A row's loss and gradient have the same bits in whatever launch it comes: alone,
where up to eight CTAs share it, or among thousands, where one CTA of fewer
threads takes it.  And the widest row with the longest list."""

import pytest
import torch

from test_gpu_distill import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def everything(S, kw, up):
    from gptq_qqq_calibration_gb300 import distill_backward, distill_forward, distill_step
    loss, d = distill_step(S, **kw)
    loss2, stats = distill_forward(S, **kw)
    return loss, loss2, stats, d, distill_backward(S, stats, grad=up, **kw)


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("dtype,vocab,start", [(torch.bfloat16, 32000, 0), (torch.bfloat16, 131037, 3),
                                               (torch.float16, 9001, 5), (torch.float32, 50257, 1)])
def test_bits_do_not_depend_on_the_launch(dtype, vocab, start, full):
    top, tau = 40, 1.25
    ld = (vocab + start + 7) // 8 * 8 + 8  # every row starts at the same place of 16 bytes
    pick = 6
    s, v, i, t = make(pick, vocab, top, dtype, vocab + start)
    lse = torch.logsumexp(t / tau, 1).float()
    gen = torch.Generator(device="cuda").manual_seed(vocab)
    # rows: from one CTA a row, several rounds of them, to few rows for all SMs
    for rows in (pick, 40, 150, 301, 470, 700, 1000, 1300, 1900, 2600, 4100):
        if rows * ld * (4 if dtype is torch.float32 else 2) > 1 << 30:
            continue
        buf = torch.randn((rows, ld), generator=gen, device="cuda", dtype=torch.float32).to(dtype)
        S = buf[:, start:start + vocab]
        V = torch.randn((rows, top), generator=gen, device="cuda")
        I = torch.randint(0, vocab, (rows, top), generator=gen, device="cuda", dtype=torch.int32)
        L = torch.logsumexp(V / tau, 1) + 0.5
        at = torch.linspace(0, rows - 1, pick).long()
        for a, r in enumerate(at.tolist()):
            S[r], V[r], I[r], L[r] = s[a].cuda(), v[a].cuda(), i[a].cuda(), lse[a].cuda()
        up = torch.ones(rows, device="cuda")
        kw = dict(top_logits=V, top_index=I, temperature=tau, teacher_lse=L if full else None)
        got = [x[at.cuda()] for x in everything(S, kw, up)]
        assert torch.equal(got[0].view(torch.int32), got[1].view(torch.int32))
        if rows == pick:
            want = got
            check(s, v, i, got[0].cpu(), got[3].cpu(), tau, lse if full else None)
            check(s, v, i, None, got[4].cpu(), tau, lse if full else None)
        for g, w in zip(got, want):
            assert torch.equal(g, w), rows
        if rows == 301:  # and each row alone
            for a, r in enumerate(at.tolist()):
                one = dict(kw, top_logits=V[r:r + 1], top_index=I[r:r + 1],
                           teacher_lse=None if not full else L[r:r + 1])
                for g, w in zip(everything(buf[r:r + 1, start:start + vocab], one, up[:1]), want):
                    assert torch.equal(g[0], w[a])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_widest_row_and_longest_list(dtype):
    from gptq_qqq_calibration_gb300 import distill_backward, distill_forward, distill_step
    vocab, top, tau = 1 << 22, 1024, 2.0
    s, v, i, t = make(2, vocab, top, dtype, 17)
    i[0, 0], i[0, 1], i[1, 5] = vocab - 1, 0, vocab - 2
    lse = torch.logsumexp(t / tau, 1).float() + 0.1
    kw = dict(top_logits=v.cuda(), top_index=i.cuda(), temperature=tau, teacher_lse=lse.cuda())
    loss, d = distill_step(s.cuda(), **kw)
    check(s, v, i, loss.cpu(), d.cpu(), tau, lse)
    loss2, stats = distill_forward(s.cuda(), **kw)
    assert torch.equal(loss, loss2)
    check(s, v, i, None, distill_backward(s.cuda(), stats, **kw).cpu(), tau, lse)
