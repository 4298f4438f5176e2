"""Gated feed-forward projections and their gradient on the GPU against a
float64 reference.

Bounds (derived per element).  u = 2^-p is half an ulp of the type, relative
(p = 8 for bf16, 11 for f16), tiny half of f16's smallest step.  A sum of K
products on the tensor cores is off by at most e(K) = (K / 16 + 8) 2^-23 times
the sum of the products' magnitudes (each 16-step may truncate once).  With
a = act(g), |act'| <= 1.13, |act''| <= 1.13 (silu and gelu both), and 2^-20
for the fast exponential and quotient:
  h  : |dg| 1.13 |u| + |a| |du| + 2^-20 |h| + u |h|
  dg : |dh| (1.13 |e_u| + 1.13 |u| |e_g| + 2^-20 |u|) + u |dg|
  du : |dh| (1.13 |e_g| + 2^-20 |a|) + u |du|
  dX, dW : the errors of dg and du through the product's magnitudes, e(K), u.
Those are worst cases; independent roundings add as squares, so the 2-norm of
the error is also held to u times the 2-norm of the result (two roundings of
at most u / sqrt 3 each: 0.82 u).
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

P = {torch.bfloat16: 8, torch.float16: 11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def make(n, d, f, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (scale * torch.randn((n, d), generator=g)).to(dtype)
    wg = (torch.randn((f, d), generator=g) / d ** 0.5).to(dtype)
    wu = (torch.randn((f, d), generator=g) / d ** 0.5).to(dtype)
    dh = (0.3 * torch.randn((n, f), generator=g)).to(dtype)
    return x, wg, wu, dh


def act64(g, kind):
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = (2 / np.pi) ** 0.5
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def reference(x, wg, wu, dh, kind):
    """(value, bound) of h, dX, dWg, dWu in float64."""
    u, tiny = 2.0 ** -P[x.dtype], TINY[x.dtype]
    X, G, U, D = (t.double() for t in (x, wg, wu, dh))
    e = lambda k: (k / 16 + 8) * 2.0 ** -23  # noqa: E731
    g, up = X @ G.T, X @ U.T
    eg, eu = e(X.shape[1]) * (X.abs() @ G.abs().T), e(X.shape[1]) * (X.abs() @ U.abs().T)
    a, da = act64(g, kind)
    h = a * up
    out = {"h": (h, 1.13 * eg * up.abs() + a.abs() * eu + eg * eu + (2.0 ** -20 + u) * h.abs() + tiny)}
    dg, du = D * up * da, D * a
    edg = D.abs() * (1.13 * eu + 1.13 * up.abs() * eg + 2.0 ** -20 * up.abs()) + u * dg.abs() + tiny
    edu = D.abs() * (1.13 * eg + 2.0 ** -20 * a.abs()) + u * du.abs() + tiny
    dx = dg @ G + du @ U
    mag = dg.abs() @ G.abs() + du.abs() @ U.abs()
    out["dx"] = dx, edg @ G.abs() + edu @ U.abs() + e(2 * G.shape[0]) * mag + u * dx.abs() + tiny
    for name, t, et in (("dwg", dg, edg), ("dwu", du, edu)):
        v = t.T @ X
        out[name] = v, et.T @ X.abs() + e(X.shape[0]) * (t.abs().T @ X.abs()) + u * v.abs() + tiny
    return out


def check(got, ref, dtype, norm=True):
    v, bound = ref
    g = got.cpu().double()
    bad = ~((g - v).abs() <= bound * 1.0001)
    assert not bad.any(), (int(bad.sum()), g[bad][:4], v[bad][:4], bound[bad][:4])
    if norm and v.norm() > 0:
        assert float((g - v).norm() / v.norm()) <= 2.0 ** -P[dtype]


SIZES = [(1, 8, 8), (1, 64, 128), (2, 72, 56), (8, 136, 264), (17, 520, 1400), (64, 256, 512), (127, 128, 136),
         (128, 512, 384), (129, 64, 72), (256, 192, 256), (257, 264, 136), (600, 1024, 640), (33, 2568, 72),
         (777, 72, 2504)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,d,f", SIZES)
def test_sizes(n, d, f, dtype):
    from gptq_qqq_calibration_gb300 import GatedFF
    for kind in ("silu", "gelu_tanh"):
        x, wg, wu, dh = make(n, d, f, dtype, 7 * n + d)
        ref = reference(x, wg, wu, dh, kind)
        op = GatedFF(d, f, train_tokens=n, dtype=dtype, activation=kind)
        X, G, U, D = (t.cuda() for t in (x, wg, wu, dh))
        check(op.forward(X, G, U), ref["h"], dtype)
        dx, dwg, dwu = op.backward(X, G, U, D)
        check(dx, ref["dx"], dtype)
        check(dwg, ref["dwg"], dtype)
        check(dwu, ref["dwu"], dtype)
        op.sync()
        op.close()


@pytest.mark.parametrize("n", [1, 2, 3, 5, 8, 9, 16, 31, 32, 33, 48, 63, 65, 96, 128, 200])
def test_few_tokens(n):
    """Token counts of decode batches, with widths that are not multiples of a tile."""
    from gptq_qqq_calibration_gb300 import GatedFF
    d, f = 1032, 1560
    x, wg, wu, dh = make(n, d, f, torch.bfloat16, n)
    op = GatedFF(d, f, dtype=torch.bfloat16)
    check(op.forward(x.cuda(), wg.cuda(), wu.cuda()), reference(x, wg, wu, dh, "silu")["h"], torch.bfloat16)
    op.sync()


@pytest.mark.parametrize("n", [1, 17, 64, 65])
def test_few_tokens_wide(n):
    """A width that gives each SM two CTAs (up to 64 tokens), and one (above)."""
    from gptq_qqq_calibration_gb300 import GatedFF
    d, f = 136, 11008
    x, wg, wu, dh = make(n, d, f, torch.bfloat16, 90 + n)
    op = GatedFF(d, f)
    check(op.forward(x.cuda(), wg.cuda(), wu.cuda()), reference(x, wg, wu, dh, "silu")["h"], torch.bfloat16)
    op.sync()


def test_many_tiles_and_repeatability():
    """More tiles than SM pairs in every contraction; the same bits each time."""
    from gptq_qqq_calibration_gb300 import GatedFF
    n, d, f = 2100, 1288, 2056
    x, wg, wu, dh = make(n, d, f, torch.bfloat16, 3)
    ref = reference(x, wg, wu, dh, "silu")
    op = GatedFF(d, f, train_tokens=n)
    args = [t.cuda() for t in (x, wg, wu, dh)]
    first = (op.forward(*args[:3]), *op.backward(*args))
    for got, k in zip(first, ("h", "dx", "dwg", "dwu")):
        check(got, ref[k], torch.bfloat16)
    again = (op.forward(*args[:3]), *op.backward(*args))
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    op.sync()


def test_wide_activations():
    """Gates far into both tails, where the exponential over- and underflows."""
    from gptq_qqq_calibration_gb300 import GatedFF
    for dtype in (torch.bfloat16, torch.float16):
        for kind in ("silu", "gelu_tanh"):
            x, wg, wu, dh = make(50, 64, 96, dtype, 9, scale=60.0)
            wu = wu * 0.05
            op = GatedFF(64, 96, train_tokens=50, dtype=dtype, activation=kind)
            ref = reference(x, wg, wu, dh, kind)
            args = [t.cuda() for t in (x, wg, wu, dh)]
            check(op.forward(*args[:3]), ref["h"], dtype)
            for got, k in zip(op.backward(*args), ("dx", "dwg", "dwu")):
                check(got, ref[k], dtype)


@pytest.mark.parametrize("n", [6, 300])
def test_bad_values_stay_in_their_rows(n):
    from gptq_qqq_calibration_gb300 import GatedFF
    x, wg, wu, dh = make(n, 128, 256, torch.bfloat16, 4)
    ref = reference(x, wg, wu, dh, "silu")
    x[2, 5] = float("nan")
    x[4, 7] = float("inf")
    op = GatedFF(128, 256, train_tokens=n)
    h = op.forward(x.cuda(), wg.cuda(), wu.cuda()).cpu()
    dx, _, _ = op.backward(x.cuda(), wg.cuda(), wu.cuda(), dh.cuda(), want_dw=False)
    keep = [r for r in range(n) if r not in (2, 4)]
    check(h[keep], tuple(t[keep] for t in ref["h"]), torch.bfloat16)
    check(dx[keep], tuple(t[keep] for t in ref["dx"]), torch.bfloat16)
    assert torch.isnan(h[2]).all() and not torch.isfinite(h[4]).all() and torch.isnan(dx[2].cpu()).all()


def test_wanted_parts_packed_weights_and_no_tokens():
    from gptq_qqq_calibration_gb300 import GatedFF
    n, d, f = 70, 160, 200
    x, wg, wu, dh = make(n, d, f, torch.bfloat16, 5)
    op = GatedFF(d, f, train_tokens=n)
    packed = torch.cat([wg, wu]).cuda()
    X, G, U, D = x.cuda(), packed[:f], packed[f:], dh.cuda()
    dx, dwg, dwu = op.backward(X, G, U, D)
    a, b, c = op.backward(X, G, U, D, want_dw=False)
    assert b is None and c is None and torch.equal(a, dx)
    a, b, c = op.backward(X, G, U, D, want_dx=False)
    assert a is None and torch.equal(b, dwg) and torch.equal(c, dwu)
    # leading dimensions are tokens
    h = op.forward(X, G, U)
    assert torch.equal(op.forward(X.view(2, 35, d), G, U).view(n, f), h)
    # no tokens: nothing for h and dX, zero weight gradients
    e = op.forward(X[:0], G, U)
    assert e.shape == (0, f)
    dx0, dwg0, dwu0 = op.backward(X[:0], G, U, D[:0])
    assert dx0.shape == (0, d) and not dwg0.any() and not dwu0.any()
    # outputs end where they should
    wide = torch.full((n + 2, f), 9.0, dtype=torch.bfloat16, device="cuda")
    op.forward(X, G, U, out=wide[1:n + 1])
    assert torch.equal(wide[1:n + 1], h) and (wide[0] == 9).all() and (wide[n + 1] == 9).all()
    op.sync()


def test_autograd_and_differences():
    from gptq_qqq_calibration_gb300 import GatedFF
    n, d, f = 40, 72, 88
    x, wg, wu, dh = make(n, d, f, torch.float16, 6)
    ref = reference(x, wg, wu, dh, "gelu_tanh")
    op = GatedFF(d, f, train_tokens=n, dtype=torch.float16, activation="gelu_tanh")
    X, G, U = (t.cuda().requires_grad_() for t in (x, wg, wu))
    (op(X, G, U) * dh.cuda()).sum().backward()
    for t, k in ((X, "dx"), (G, "dwg"), (U, "dwu")):
        check(t.grad, ref[k], torch.float16)
    # directional differences of the float64 value
    gen = torch.Generator().manual_seed(0)
    val = lambda a, b, c: float((act64(a @ b.T, "gelu_tanh")[0] * (a @ c.T) * dh.double()).sum())  # noqa: E731
    base = [t.double() for t in (x, wg, wu)]
    for k, (t, name) in enumerate(((X, "dx"), (G, "dwg"), (U, "dwu"))):
        e = torch.randn(base[k].shape, generator=gen, dtype=torch.float64)
        hi = [b + 1e-4 * e if j == k else b for j, b in enumerate(base)]
        lo = [b - 1e-4 * e if j == k else b for j, b in enumerate(base)]
        diff = (val(*hi) - val(*lo)) / 2e-4
        got = float((t.grad.cpu().double() * e).sum())
        assert abs(got - diff) <= float((ref[name][1] * e.abs()).sum()) + 1e-5 * abs(diff)
    # only what needs a gradient gets one
    X2 = x.cuda().requires_grad_()
    op(X2, G.detach(), U.detach()).sum().backward()
    assert X2.grad is not None


def test_streams_share_one_workspace():
    """Backward calls of one handle on different streams do not mix."""
    from gptq_qqq_calibration_gb300 import GatedFF
    n, d, f = 1500, 512, 1024
    op = GatedFF(d, f, train_tokens=n)
    sets = [[t.cuda() for t in make(n, d, f, torch.bfloat16, 20 + k)] for k in range(4)]
    want = [op.backward(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = [op.backward(*s, stream=st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    op.sync()


def test_graph_capture():
    from gptq_qqq_calibration_gb300 import GatedFF
    n, d, f = 100, 256, 512
    op = GatedFF(d, f, train_tokens=n)
    X, G, U, D = (t.cuda() for t in make(n, d, f, torch.bfloat16, 30))
    want = (op.forward(X, G, U), *op.backward(X, G, U, D))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        op.forward(X, G, U), op.backward(X, G, U, D)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = (op.forward(X, G, U), *op.backward(X, G, U, D))
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_rows_past_32_bit_offsets():
    """More than 2^32 elements of h."""
    from gptq_qqq_calibration_gb300 import GatedFF
    n, d, f = 400000, 64, 11008
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn((n, d), generator=g, device="cuda").bfloat16()
    _, wg, wu, _ = make(1, d, f, torch.bfloat16, 40)
    op = GatedFF(d, f)
    h = op.forward(X, wg.cuda(), wu.cuda())
    rows = [0, 195000, 195083, 195084, 390168, n - 1]
    x = X[rows].cpu()
    check(h[rows], reference(x, wg, wu, torch.zeros((len(rows), f), dtype=torch.bfloat16), "silu")["h"],
          torch.bfloat16)
    op.sync()


def test_feeds_the_hessian():
    """h goes into the calibration Hessian of the down projection as it comes."""
    from gptq_qqq_calibration_gb300 import GatedFF, Hessian
    n, d, f = 300, 256, 384
    x, wg, wu, _ = make(n, d, f, torch.bfloat16, 50)
    op = GatedFF(d, f)
    hess = Hessian(f)
    h = op.forward(x.cuda(), wg.cuda(), wu.cuda())
    hess.add_batch(h)
    H, _ = hess.materialize(0.0)
    hess.sync()
    hd = h.cpu().double()
    want = 2.0 / n * hd.T @ hd
    assert float((H.cpu().double() - want).abs().max()) <= 5e-5 * float(want.diagonal().mean())


def test_timeout_is_reported_and_recovers():
    """A wait limit of zero makes the kernels give up; the status says so, and
    the handle works again afterwards."""
    from gptq_qqq_calibration_gb300 import GatedFF, HessError
    from gptq_qqq_calibration_gb300.gated_ff import gated_ff_set_timeout
    n, d, f = 300, 512, 512
    op = GatedFF(d, f, train_tokens=n)
    X, G, U, D = (t.cuda() for t in make(n, d, f, torch.bfloat16, 60))
    want = op.forward(X, G, U)
    op.sync()
    gated_ff_set_timeout(op.handle, 0)
    op.forward(X, G, U)
    with pytest.raises(HessError, match="TIMEOUT"):
        op.sync()
    gated_ff_set_timeout(op.handle, 2_000_000_000)
    assert torch.equal(op.forward(X, G, U), want)
    op.sync()


def test_few_tokens_on_streams_and_after_a_timeout():
    """Calls of few tokens share the handle's workspace: on several streams they
    do not mix, and a call that gave up leaves nothing behind once it is
    reported."""
    from gptq_qqq_calibration_gb300 import GatedFF, HessError
    from gptq_qqq_calibration_gb300.gated_ff import gated_ff_set_timeout
    d, f = 2048, 3000
    op = GatedFF(d, f)
    sets = [[t.cuda() for t in make(n, d, f, torch.bfloat16, 70 + n)[:3]] for n in (1, 20, 90, 128)]
    want = [op.forward(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [op.forward(*s, stream=st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    op.sync()
    gated_ff_set_timeout(op.handle, 0)
    op.forward(*sets[1])
    with pytest.raises(HessError, match="TIMEOUT"):
        op.sync()
    gated_ff_set_timeout(op.handle, 2_000_000_000)
    assert all(torch.equal(op.forward(*s), w) for s, w in zip(sets, want))
    op.sync()


def test_refusals():
    from gptq_qqq_calibration_gb300 import GatedFF, HessError
    from gptq_qqq_calibration_gb300 import _lib
    x, wg, wu, dh = make(16, 64, 128, torch.bfloat16, 1)
    X, G, U, D = (t.cuda() for t in (x, wg, wu, dh))
    op = GatedFF(64, 128, train_tokens=8)
    for bad in (lambda: op.forward(x, G, U), lambda: op.forward(X.half(), G, U), lambda: op.forward(X, G.t(), U),
                lambda: op.forward(X[:, :32], G, U), lambda: op.forward(X, G[:64], U),
                lambda: op.forward(X, G, U, out=torch.empty((3, 128), dtype=torch.bfloat16, device="cuda")),
                lambda: op.backward(X, G, U, D[:3]), lambda: GatedFF(64, 128, activation="relu"),
                lambda: GatedFF(64, 128, dtype=torch.float64)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: GatedFF(60, 128), lambda: GatedFF(64, 65544), lambda: GatedFF(0, 128),
                lambda: GatedFF(64, 128, dtype=torch.float32), lambda: GatedFF(64, 128, train_tokens=-1),
                lambda: op.backward(X, G, U, D)):  # 16 tokens, workspace for 8
        with pytest.raises(HessError):
            bad()
    flat = torch.zeros(64 * 16 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(HessError):  # not 16-byte aligned
        op.forward(flat[1:64 * 16 + 1].view(16, 64), G, U)
    lib = _lib.load()
    out = torch.empty((16, 128), dtype=torch.bfloat16, device="cuda")
    hostbuf = torch.zeros(16 * 128, dtype=torch.bfloat16)
    args = [op.handle, X.data_ptr(), 16, G.data_ptr(), U.data_ptr(), out.data_ptr(), None]
    for at in (1, 3, 4, 5):
        bad = list(args)
        bad[at] = hostbuf.data_ptr()
        assert lib.gated_ff_forward(*bad) == _lib.HESS_ERR_INVALID
        bad[at] = None
        assert lib.gated_ff_forward(*bad) == _lib.HESS_ERR_INVALID
    assert lib.gated_ff_forward(*args) == _lib.HESS_OK
    op.sync()
