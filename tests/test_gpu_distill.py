"""Distillation loss and gradient on the GPU against the float64 oracle.

Bounds (derived from the arithmetic, per element).  With eps = 1e-6 (2 + R),
R the largest |logit| / tau: the exponent s k2 - M2 is one fp32 FMA of a k2
rounded to fp32 (errors 2^-24 of the exponent and of s k2, both at most about
R log2 e), ex2 is good to 2^-22, and sums of a row add a few 2^-24:
  loss     : w tau^2 (eps (1 + p_r / q_r dependence below) + 2^-23 |L|)
  gradient : half an ulp of the output type of the reference, plus
             w tau eps (q + p) in the list, and outside it
             w tau eps (q + p_r q / q_r) + w tau 3e-7 (2 + R) q / q_r
             (the last: p_r = 1 - sum p has an absolute error).
"""

import ctypes

import numpy as np
import pytest
import torch

from oracle.distill_oracle import distill_row

pytestmark = pytest.mark.gpu

# half an ulp, relative: 2^-p for p significand bits (8, 11, 24)
ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-38}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def make(rows, vocab, top, dtype, seed, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    s = (scale * torch.randn((rows, vocab), generator=g)).to(dtype)
    t = s.float() + 0.8 * torch.randn((rows, vocab), generator=g)
    k = min(top, vocab)
    v, i = torch.topk(t, k, dim=1)
    if k < top:  # the rest of the list is empty
        v = torch.cat([v, torch.zeros(rows, top - k)], 1)
        i = torch.cat([i, torch.full((rows, top - k), -1)], 1)
    return s, v, i.to(torch.int32), t.double()


def check(s, v, i, loss, grad, tau, lse=None, w=None, up=None):
    """Compares GPU results (host tensors) with the oracle, row by row."""
    sn = s.double().numpy()
    for r in range(s.shape[0]):
        wt = 1.0 if w is None else float(w[r])
        o = distill_row(sn[r], v[r].double().numpy(), i[r].numpy(), tau, None if lse is None else float(lse[r]), wt)
        fin = sn[r][np.abs(sn[r]) < 1e30]  # masks of the type's lowest value carry nothing
        tf = v[r].double().numpy()
        tf = tf[np.isfinite(tf)]
        R = max(np.abs(fin).max() if fin.size else 0.0, np.abs(tf).max() if tf.size else 0.0) / tau
        eps = 1e-6 * (2 + R)
        if loss is not None:
            got = float(loss[r])
            if np.isnan(o["loss"]) or np.isinf(o["loss"]):
                assert np.isnan(got) if np.isnan(o["loss"]) else got == o["loss"], (r, got, o["loss"])
            else:
                ratio = np.log(o["p_rest"] / o["q_rest"]) if o["p_rest"] > 0 else 0.0
                tol = abs(wt) * tau ** 2 * eps * (1 + abs(ratio)) + 2.0 ** -23 * abs(o["loss"])
                assert abs(got - o["loss"]) <= tol, (r, got, o["loss"], tol)
        if grad is not None:
            g = grad[r].double().numpy()
            gs = abs(wt) * tau
            ref = o["grad"]
            if up is not None:
                gs, ref = gs * abs(float(up[r])), ref * float(up[r])
            if np.isnan(ref).any():
                assert np.isnan(g).all(), r
                continue
            over = o["q"] / o["q_rest"] if o["p_rest"] > 0 and o["q_rest"] > 0 else 0.0 * o["q"]
            tol = gs * np.where(o["listed"], eps * (o["q"] + o["p"]),
                                eps * (o["q"] + o["p_rest"] * over) + 3e-7 * (2 + R) * over)
            tol = tol + ULP[grad.dtype] * np.abs(ref) * 1.01 + TINY[grad.dtype]
            bad = ~(np.abs(g - ref) <= tol)
            assert not bad.any(), (r, np.flatnonzero(bad)[:5], g[bad][:5], ref[bad][:5], tol[bad][:5])


def run_all(s, v, i, tau, lse=None, w=None, up=None):
    from gptq_qqq_calibration_gb300 import distill_backward, distill_forward, distill_step
    c = lambda x: None if x is None else x.cuda()  # noqa: E731
    kw = dict(temperature=tau, teacher_lse=c(lse), weights=c(w))
    S, V, I = s.cuda(), v.cuda(), i.cuda()
    loss1, d1 = distill_step(S, V, I, **kw)
    loss2, stats = distill_forward(S, V, I, **kw)
    d2 = distill_backward(S, stats, V, I, grad=c(up), **kw)
    torch.cuda.synchronize()
    assert torch.equal(loss1.view(torch.int32), loss2.view(torch.int32))
    check(s, v, i, loss1.cpu(), d1.cpu(), tau, lse, w)
    check(s, v, i, None, d2.cpu(), tau, lse, w, up)
    return loss1.cpu(), d1.cpu(), d2.cpu()


SIZES = [(1, 1, 1), (3, 7, 2), (2, 16, 16), (5, 33, 40), (7, 257, 5), (2, 1000, 1000), (4, 4099, 17), (3, 40000, 64),
         (9, 65536, 128), (2, 140001, 33)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,vocab,top", SIZES)
def test_sizes(rows, vocab, top, dtype):
    s, v, i, t = make(rows, vocab, top, dtype, rows * 1000 + vocab)
    g = torch.Generator().manual_seed(1)
    w = torch.rand(rows, generator=g) - 0.2
    up = torch.rand(rows, generator=g) - 0.5
    run_all(s, v, i, 1.0)
    tau = 1.7
    run_all(s, v, i, tau, torch.logsumexp(t / tau, 1).float(), w, up)


def test_row_longer_than_a_cluster_holds():
    """3.2 MB rows: every CTA goes through its slice in pieces, twice."""
    s, v, i, t = make(2, 800003, 50, torch.float32, 5)
    run_all(s, v, i, 2.0, torch.logsumexp(t / 2.0, 1).float())


@pytest.mark.parametrize("tau", [0.25, 4.0])
@pytest.mark.parametrize("top_dtype,index_dtype", [(torch.float32, torch.int64), (torch.bfloat16, torch.int32),
                                                   (torch.float16, torch.int64)])
def test_list_types(top_dtype, index_dtype, tau):
    s, v, i, t = make(6, 5000, 20, torch.bfloat16, 11)
    run_all(s, v.to(top_dtype), i.to(index_dtype), tau, torch.logsumexp(t / tau, 1).float() + 0.01)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_masked_rows_and_empty_slots(dtype):
    """Rows without weight or without teacher entries give zeros whatever
    their logits hold; lists that end early, slots of -inf."""
    s, v, i, t = make(8, 999, 12, dtype, 21)
    lse = torch.logsumexp(t, 1).float()
    w = torch.ones(8)
    w[1] = w[4] = 0.0
    s[1] = float("nan")
    s[4, 5] = float("inf")
    i[2] = -1
    s[2] = float("nan")
    v[3] = -float("inf")
    i[5, 3:] = -7
    v[6, ::2] = -float("inf")
    for l in (None, lse):
        loss, d, d2 = run_all(s, v, i, 1.5, l, w, torch.ones(8))
        for r in (1, 2, 3, 4):
            assert float(loss[r]) == 0.0 and not d[r].any() and not d2[r].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,vocab,top,tau,scale", [(6, 62652, 7, 3.0, 0.5), (5, 33001, 3, 1.0, 0.3),
                                                      (4, 9000, 40, 2.0, 1.0), (3, 140001, 16, 4.0, 2.0)])
def test_little_mass_in_the_list(rows, vocab, top, tau, scale, dtype):
    """Loss and gradients are small against the masses outside the list, which are
    nearly one on both sides: they keep the accuracy of the masses P and Q in it.

    Bounds, with eps as above: p and q of listed columns have relative errors of eps.
    The loss is sum p log(p / q) + (1 - P) (log1p(-P) - log1p(-Q)), whose derivatives
    by the listed p and q are at most |log(p / q)| + 1 + |log((1 - P) / (1 - Q))| and
    p / q + 1 / (1 - Q): errors of eps (P (3 + max |log(p / q)|) + 2 Q).  Outside the
    list the gradient is w tau (P - Q) q / q_rest: eps 2 (P + Q) q / q_rest.
    """
    s, v, i, t = make(rows, vocab, top, dtype, vocab + top, scale)
    lse = torch.logsumexp(t / tau, 1).float()
    loss, d1, d2 = run_all(s, v, i, tau, lse)
    for r in range(rows):
        o = distill_row(s[r].double().numpy(), v[r].double().numpy(), i[r].numpy(), tau, float(lse[r]))
        inside = o["listed"]
        P, Q = o["p"][inside].sum(), o["q"][inside].sum()
        assert P < 0.5 and Q < 0.5
        eps = 1e-6 * (2 + max(s[r].float().abs().max().item(), v[r].abs().max().item()) / tau)
        ratio = np.abs(np.log(o["p"][inside] / o["q"][inside])).max()
        tol = tau ** 2 * eps * (P * (3 + ratio) + 2 * Q) + 2.0 ** -22 * abs(o["loss"])
        assert abs(float(loss[r]) - o["loss"]) <= tol, (r, float(loss[r]), o["loss"], tol)
        ref = o["grad"]
        tol = tau * eps * np.where(inside, o["q"] + o["p"], 2 * (P + Q) * o["q"] / o["q_rest"])
        tol = tol + ULP[dtype] * np.abs(ref) * 1.01 + TINY[dtype]
        for d in (d1, d2):
            bad = ~(np.abs(d[r].double().numpy() - ref) <= tol)
            assert not bad.any(), (r, np.flatnonzero(bad)[:5], d[r][torch.from_numpy(bad)][:5], ref[bad][:5], tol[bad][:5])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinite_and_nan_logits(dtype):
    """-inf columns (a padded vocabulary) carry no probability; a column the
    teacher wants but the student masks gives an infinite loss; NaN and +inf
    stay in their rows; an index past the vocabulary makes its row NaN."""
    s, v, i, t = make(7, 3000, 10, dtype, 31)
    s[0, 2000:] = -float("inf")
    i[0] = torch.arange(10, dtype=torch.int32) * 190
    s[1, int(i[1, 4])] = -float("inf")
    i[2, 3] = 3000
    s[3, 17] = float("nan")
    s[4, 18] = float("inf")
    lse = torch.logsumexp(t, 1).float()
    from gptq_qqq_calibration_gb300 import distill_backward, distill_forward, distill_step
    for l in (None, lse):
        kw = dict(teacher_lse=None if l is None else l.cuda())
        loss, d = distill_step(s.cuda(), v.cuda(), i.cuda(), **kw)
        _, stats = distill_forward(s.cuda(), v.cuda(), i.cuda(), **kw)
        d2 = distill_backward(s.cuda(), stats, v.cuda(), i.cuda(), **kw)
        for g in (d.cpu(), d2.cpu()):
            assert torch.isnan(loss[3]) and torch.isnan(loss[4])
            assert torch.isnan(g[3]).all() and torch.isnan(g[4]).all()
            keep = [0, 1, 2, 5, 6]
            check(s[keep], v[keep], i[keep], loss.cpu()[keep], g[keep], 1.0, None if l is None else l[keep])
            assert torch.isinf(loss[1]) and torch.isnan(loss[2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_lowest_value_masks_and_wide_logits(dtype):
    """Columns masked with the type's lowest value, logits hundreds apart, and
    a mass outside the list that underflows next to the listed columns."""
    s, v, i, t = make(4, 2048, 8, dtype, 41)
    s[0, 1000:] = torch.finfo(dtype).min
    i[0] = torch.arange(8, dtype=torch.int32) * 3
    s[1] = (s[1].float() * 100).to(dtype)
    s[2] = s[2] - 500
    s[2, i[2].long()] = 1.0  # q outside the list is about e^-500
    lse = torch.logsumexp(t, 1).float()
    # values this far apart: the exponent itself carries 2^-24 of its size
    run_all(s, v, i, 1.0, None)
    run_all(s[2:], v[2:], i[2:], 1.0, lse[2:])


def test_duplicate_columns():
    s, v, i, t = make(3, 600, 16, torch.float32, 51)
    i[0, 5] = i[0, 2]
    i[1, 15] = i[1, 0]
    i[1, 7] = i[1, 0]
    i[2, :] = 9
    a = run_all(s, v, i, 1.0, None)
    b = run_all(s, v, i, 1.0, torch.logsumexp(t, 1).float() + 3.0)
    c = run_all(s, v, i, 1.0, None)
    assert all(torch.equal(x, y) for x, y in zip(a, c)) and not torch.equal(a[0], b[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,start,opad", [(7, 3, 0), (8, 0, 8), (1, 1, 1), (5, 0, 2)])
def test_strides_alignment_and_in_place(dtype, pad, start, opad):
    """Rows of a wider buffer at any element offset; outputs with another
    stride; the gradient written over the logits.  Nothing around the rows
    changes."""
    from gptq_qqq_calibration_gb300 import distill_backward, distill_forward, distill_step
    rows, vocab = 5, 1237
    s, v, i, t = make(rows, vocab, 9, dtype, 61)
    lse = torch.logsumexp(t, 1).float()
    V, I, L = v.cuda(), i.cuda(), lse.cuda()
    wide = torch.full((rows, vocab + pad), 77.0, dtype=dtype, device="cuda")
    wide[:, start:start + vocab] = s.cuda()
    S = wide[:, start:start + vocab]
    owide = torch.full((rows, vocab + opad), 55.0, dtype=dtype, device="cuda")
    O = owide[:, opad:]
    loss, d = distill_step(S, V, I, teacher_lse=L, out=O)
    check(s, v, i, loss.cpu(), d.cpu(), 1.0, lse)
    assert (owide[:, :opad] == 55).all() and (wide[:, :start] == 77).all() and (wide[:, start + vocab:] == 77).all()
    loss2, stats = distill_forward(S, V, I, teacher_lse=L)
    want = distill_backward(S, stats, V, I, teacher_lse=L)
    assert torch.equal(loss, loss2)
    save = wide.clone()
    distill_backward(S, stats, V, I, teacher_lse=L, out=S)
    assert torch.equal(S, want)
    wide.copy_(save)
    loss3, _ = distill_step(S, V, I, teacher_lse=L, out=S)
    assert torch.equal(S, d) and torch.equal(loss3, loss)
    assert (wide[:, :start] == 77).all() and (wide[:, start + vocab:] == 77).all()


def test_autograd_and_differences():
    """distill_loss under autograd equals the one-pass gradient's formula and
    the differences of the float64 loss."""
    from gptq_qqq_calibration_gb300 import distill_loss
    s, v, i, t = make(4, 300, 6, torch.float32, 71)
    lse = torch.logsumexp(t, 1).float()
    w = torch.tensor([0.5, 1.0, 0.0, 2.0])
    up = torch.tensor([1.0, -2.0, 3.0, 0.25])
    S = s.cuda().requires_grad_()
    loss = distill_loss(S, v.cuda(), i.cuda(), 1.3, lse.cuda(), w.cuda())
    (loss * up.cuda()).sum().backward()
    g = S.grad.cpu().double().numpy()
    check(s, v, i, loss.detach().cpu(), S.grad.cpu(), 1.3, lse, w, up)
    h = 1e-4
    rng = np.random.default_rng(0)
    for r in range(4):
        for _ in range(4):
            e = rng.normal(size=300)
            f = lambda x: distill_row(x, v[r].double().numpy(), i[r].numpy(), 1.3, float(lse[r]), float(w[r]))["loss"]  # noqa: E731
            x = s[r].double().numpy()
            d = (f(x + h * e) - f(x - h * e)) / (2 * h) * float(up[r])
            assert abs(d - (g[r] * e).sum()) <= 1e-5 * (1 + abs(d)) * (abs(float(w[r] * up[r])) + 0.1)
    T = s.cuda().requires_grad_()
    distill_loss(T, v.cuda(), i.cuda()).mean().backward()  # an expanded upstream gradient
    check(s, v, i, None, T.grad.cpu(), 1.0, None, None, torch.full((4,), 0.25))


def test_streams_and_repeatability():
    from gptq_qqq_calibration_gb300 import distill_step
    s, v, i, _ = make(64, 33000, 40, torch.bfloat16, 81)
    S, V, I = s.cuda(), v.cuda(), i.cuda()
    want = distill_step(S, V, I)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [distill_step(S, V, I, stream=st) for st in streams]
    torch.cuda.synchronize()
    for g in got:
        assert torch.equal(g[0], want[0]) and torch.equal(g[1], want[1])


def test_no_rows_and_leading_dimensions():
    from gptq_qqq_calibration_gb300 import distill_forward, distill_step
    e = torch.empty((0, 50), device="cuda")
    loss, d = distill_step(e, torch.empty((0, 4), device="cuda"), torch.empty((0, 4), dtype=torch.int32, device="cuda"))
    assert loss.shape == (0,) and d.shape == (0, 50)
    s, v, i, _ = make(6, 77, 3, torch.float32, 91)
    a = distill_forward(s.cuda(), v.cuda(), i.cuda())[0]
    b = distill_forward(s.cuda().view(2, 3, 77), v.cuda().view(2, 3, 3), i.cuda().view(2, 3, 3))[0]
    assert torch.equal(a, b)


def test_rows_past_32_bit_offsets():
    """More than 2^32 elements of logits: the last rows are as right as the first."""
    from gptq_qqq_calibration_gb300 import distill_step
    rows, vocab = 33000, 131072
    S = torch.zeros((rows, vocab), dtype=torch.bfloat16, device="cuda")
    pick = [0, 16384, 32767, 32768, rows - 1]
    s, v, i, _ = make(len(pick), vocab, 8, torch.bfloat16, 101)
    V = torch.zeros((rows, 8), device="cuda")
    I = torch.full((rows, 8), -1, dtype=torch.int32, device="cuda")
    for a, r in enumerate(pick):
        S[r], V[r], I[r] = s[a].cuda(), v[a].cuda(), i[a].cuda()
    loss, d = distill_step(S, V, I)
    check(s, v, i, loss[pick].cpu(), d[pick].cpu(), 1.0)
    assert not d[1:16384].any() and not d[32769:rows - 1].any()


def test_refusals():
    from gptq_qqq_calibration_gb300 import HessError, distill_forward, distill_step
    from gptq_qqq_calibration_gb300 import _lib
    s, v, i, _ = make(4, 100, 5, torch.bfloat16, 1)
    S, V, I = s.cuda(), v.cuda(), i.cuda()
    with pytest.raises(ValueError):
        distill_forward(s, V, I)  # host tensor
    with pytest.raises(ValueError):
        distill_forward(S.double(), V, I)
    with pytest.raises(ValueError):
        distill_forward(S.t(), V, I)
    with pytest.raises(ValueError):
        distill_forward(S, V, I.to(torch.int16))
    with pytest.raises(ValueError):
        distill_forward(S, V[:, :3], I)
    with pytest.raises(ValueError):
        distill_forward(S, V, I, weights=torch.ones(3, device="cuda"))
    with pytest.raises(ValueError):
        distill_step(S, V, I, out=torch.empty((4, 100), device="cuda"))
    for tau in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(HessError):
            distill_forward(S, V, I, temperature=tau)
    with pytest.raises(HessError):
        distill_forward(S, torch.zeros((4, 1025), device="cuda"), torch.zeros((4, 1025), dtype=torch.int32, device="cuda"))
    buf = torch.zeros(1000, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(HessError):  # overlapping, but not the logits themselves
        distill_step(buf[:400].view(4, 100), V, I, out=buf[8:408].view(4, 100))
    # host memory at the C entry is an argument error, not a fault
    lib = _lib.load()
    loss, stats = torch.empty(4, device="cuda"), torch.empty((4, 8), device="cuda")
    args = [S.data_ptr(), 100, 4, 100, 0, V.data_ptr(), 1, I.data_ptr(), 4, 5, None, None, 1.0, loss.data_ptr(),
            stats.data_ptr(), None]
    hostbuf = torch.zeros(4000)
    for at in (0, 5, 7, 13, 14):
        bad = list(args)
        bad[at] = hostbuf.data_ptr()
        assert lib.distill_forward(*bad) == _lib.HESS_ERR_INVALID
    assert lib.distill_forward(*args) == _lib.HESS_OK
    torch.cuda.synchronize()
