"""The 8-bit integer linear layer on the GPU.

Forward is compared bit for bit: the integer sum (64-bit on the CPU) is rounded to
float32, scaled by the float32 product of the two scales, and rounded to the type.

Gradients are compared with 64-bit products of dY and the restored values W^ and X^
(code times scale in float32, rounded to the type by the CPU, which is what the
header promises).  A sum of K products on the tensor cores is off by at most
e(K) = (K / 16 + 8) 2^-23 times the sum of the products' magnitudes (each 16-step
may truncate once, pieces are added in fp32), and the result is rounded once, by
at most u = eps / 2 of itself.  Independent errors add as squares: the 2-norm of
the error is held to u times that of the result.
"""

import pytest
import torch

from test_gpu_rows8 import formula, values

pytestmark = pytest.mark.gpu

# tokens, d, f: what the layout has at 76 pairs ("split": tiles in several pieces, "whole": whole
# tiles before them, "rows": fewer than 128 weight rows per CTA, "tokens": several tiles of tokens)
LAYOUTS = {
    (33, 4096, 1400): "split rows",
    (37, 11008, 4096): "split",
    (24, 4096, 11008): "rows",
    (20, 65536, 2048): "split",
    (300, 40000, 2056): "split rows tokens",
    (1000, 8192, 4096): "split whole tokens",
    (1500, 1040, 2048): "tokens",
}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def rows8(codes, scale, group=0):
    from gptq_qqq_calibration_gb300 import Rows8
    return Rows8(codes.cuda(), scale.cuda(), group)


def make(n, d, f, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, d), generator=g)
    x[:, torch.rand(d, generator=g) < 0.02] *= 10.0
    x[torch.rand(n, generator=g) < 0.1] = 0.0
    w = formula(torch.randn((f, d), generator=g) / d ** 0.5, 0)
    dy = 0.3 * torch.randn((n, f), generator=g)
    return x.to(dtype), w, dy.to(dtype)


def product(xq, xs, wq, ws, dtype):
    """Bits of y."""
    total = (xq.double() @ wq.double().T).float()  # exact below 2^53, rounded once
    return (total * (xs[:, None] * ws[None, :])).to(dtype)


def same(a, b):
    return torch.equal(torch.nan_to_num(a.cpu().float(), 7.25), torch.nan_to_num(b.float(), 7.25))


def check_forward(n, d, f, dtype, seed):
    from gptq_qqq_calibration_gb300 import Int8Linear, quantize_rows
    x, (wq, ws), _ = make(n, d, f, dtype, seed)
    xq, xs = formula(x, 0)
    want = product(xq, xs, wq, ws, dtype)
    op = Int8Linear(d, f, tokens=n, dtype=dtype)
    weight = rows8(wq, ws)
    X = x.cuda()
    assert same(op.forward(X, weight), want)
    assert same(op.forward(quantize_rows(X), weight), want)
    op.sync()
    op.close()


SIZES = [(1, 16, 8), (1, 32, 136), (2, 144, 264), (3, 4096, 520), (4, 1040, 1400), (5, 528, 264), (8, 4096, 2048),
         (9, 16, 8), (9, 144, 24), (16, 528, 1400), (17, 2064, 264), (31, 128, 520), (64, 1040, 4104),
         (128, 4096, 1032), (191, 256, 136), (192, 512, 264), (193, 1024, 520), (385, 2064, 520), (700, 528, 1400),
         (8, 8192, 72), (8, 8208, 72), (4, 16384, 40), (4, 16400, 40), (2, 32768, 24), (2, 32784, 24), (1, 65536, 16),
         (20, 65536, 16), (18, 4096, 9728), (24, 1040, 4872), (32, 4096, 4864), (27, 2048, 4872), (17, 4112, 264)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,d,f", SIZES)
def test_forward_sizes(n, d, f, dtype):
    check_forward(n, d, f, dtype, n + d + f)


@pytest.mark.parametrize("n,d,f", list(LAYOUTS))
def test_forward_layouts(n, d, f):
    check_forward(n, d, f, torch.bfloat16, n + 1)


@pytest.mark.parametrize("n", list(range(1, 13)) + [15, 17, 23, 24, 25, 31, 32, 33, 47, 48, 49, 95, 97])
def test_forward_token_counts(n):
    check_forward(n, 1040, 1560, torch.bfloat16, 500 + n)


@pytest.mark.parametrize("n", [1, 8, 9, 200])
@pytest.mark.parametrize("d", [1024, 1040, 11008])
def test_sums_that_float32_does_not_hold(n, d):
    """Codes at their ends: partial sums far beyond 2^24 that cancel to small numbers."""
    from gptq_qqq_calibration_gb300 import Int8Linear
    f = 264
    g = torch.Generator().manual_seed(d + n)
    xq = torch.full((n, d), -128, dtype=torch.int8)
    wq = torch.full((f, d), -128, dtype=torch.int8)
    wq[1::4] = 127
    wq[2::4, d // 2:] = 127  # half of the sum up, half down
    wq[3::4] = torch.randint(-128, 128, (len(range(3, f, 4)), d), generator=g).to(torch.int8)
    xq[n // 2:] = torch.randint(-128, 128, (n - n // 2, d), generator=g).to(torch.int8)
    for scale in (1.0, 2.0 ** -12):
        xs, ws = torch.full((n,), scale), torch.full((f,), 1.0)
        op = Int8Linear(d, f, tokens=n, dtype=torch.bfloat16)
        got = op.forward(rows8(xq, xs), rows8(wq, ws))
        op.sync()
        assert same(got, product(xq, xs, wq, ws, torch.bfloat16))
    # differences of equal rows are exact: y of q and of q with one code changed by 1 differ by one code
    one = xq.clone()
    one[:, 5] = one[:, 5] ^ 1
    xs = torch.full((n,), 2.0 ** -8)
    ws = torch.full((f,), 2.0 ** -8)
    op = Int8Linear(d, f, tokens=n, dtype=torch.float16)
    assert same(op.forward(rows8(one, xs), rows8(wq, ws)), product(one, xs, wq, ws, torch.float16))
    op.sync()


@pytest.mark.parametrize("n", [2, 40])
def test_rows_of_zeros_and_not_finite(n):
    from gptq_qqq_calibration_gb300 import Int8Linear
    d, f = 272, 136
    x, (wq, ws), _ = make(n, d, f, torch.bfloat16, 9)
    x[0] = 0.0
    x[1, 7] = float("inf")
    ws[3] = 0.0
    op = Int8Linear(d, f, tokens=n)
    got = op.forward(x.cuda(), rows8(wq, ws)).cpu()
    op.sync()
    assert (got[0] == 0).all() and got[1].isnan().all()
    assert same(got, product(*formula(x, 0), wq, ws, torch.bfloat16))


def check(got, want, bound, dtype):
    u = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    g = got.cpu().double()
    bad = ~((g - want).abs() <= (bound + u * want.abs() + tiny) * 1.0001)
    assert not bad.any(), (int(bad.sum()), g[bad][:4], want[bad][:4])
    if want.norm() > 0:
        assert float((g - want).norm() / want.norm()) <= u


def check_backward(n, d, f, dtype, group, seed):
    from gptq_qqq_calibration_gb300 import Int8Linear
    x, (wq, ws), dy = make(n, d, f, dtype, seed)
    xq, xs = formula(x, group)
    w64, x64, d64 = values(wq, ws, 0, dtype).double(), values(xq, xs, group, dtype).double(), dy.double()
    e = lambda k: (k / 16 + 8) * 2.0 ** -23  # noqa: E731
    op = Int8Linear(d, f, tokens=0, train_tokens=n, dtype=dtype)
    dx, dw = op.backward(dy.cuda(), rows8(xq, xs, group), rows8(wq, ws))
    op.sync()
    check(dx, d64 @ w64, e(f) * (d64.abs() @ w64.abs()), dtype)
    check(dw, d64.T @ x64, e(n) * (d64.abs().T @ x64.abs()), dtype)
    one, none = op.backward(dy.cuda(), rows8(xq, xs, group), rows8(wq, ws), want_dw=False)
    assert none is None and torch.equal(one, dx)
    none, one = op.backward(dy.cuda(), rows8(xq, xs, group), rows8(wq, ws), want_dx=False)
    assert none is None and torch.equal(one, dw)
    op.sync()
    op.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,d,f", [(1, 16, 8), (2, 144, 264), (17, 528, 1400), (64, 256, 512), (129, 64, 72),
                                   (203, 528, 1400), (257, 272, 136), (600, 1024, 640), (777, 80, 2504),
                                   (1100, 2064, 520)])
def test_backward_sizes(n, d, f, dtype):
    check_backward(n, d, f, dtype, 0, n + d)
    check_backward(n, d, f, dtype, (32, 64, 128, 256)[n % 4], n + d + 1)


def test_gradients_by_differences():
    """The layer is linear in the restored values: a step of one code in one place of X or
    W changes sum(dY y) by the gradient there times the scale."""
    from gptq_qqq_calibration_gb300 import Int8Linear
    n, d, f = 24, 144, 136
    x, (wq, ws), dy = make(n, d, f, torch.bfloat16, 77)
    xq, xs = formula(x, 0)
    op = Int8Linear(d, f, tokens=n, train_tokens=n)
    dx, dw = (t.cpu().double() for t in op.backward(dy.cuda(), rows8(xq, xs), rows8(wq, ws)))
    op.sync()
    u = torch.finfo(torch.bfloat16).eps / 2

    def objective(xc, wc):  # the forward's formula in 64 bits, on which the kernel is exact up to a rounding
        return (dy.double() * ((xc.double() @ wc.double().T) * xs.double()[:, None] * ws.double())).sum()

    base = objective(xq, wq)
    mag_x = dy.double().abs() @ values(wq, ws, 0, torch.bfloat16).double().abs()
    mag_w = dy.double().abs().T @ values(xq, xs, 0, torch.bfloat16).double().abs()
    for k in range(12):
        t, c, i = k % n, (7 * k) % f, (31 * k) % d
        other = xq.clone().double()
        other[t, i] += 1
        step = float(objective(other, wq) - base)
        # W^ rounded (u of every term), dX rounded (u), fp32 sums
        assert abs(step - float(dx[t, i] * xs[t].double())) <= 2.1 * u * float(mag_x[t, i] * xs[t].double()) + 1e-9
        other = wq.clone().double()
        other[c, i] += 1
        step = float(objective(xq, other) - base)
        assert abs(step - float(dw[c, i] * ws[c].double())) <= 2.1 * u * float(mag_w[c, i] * ws[c].double()) + 1e-9


def test_no_tokens():
    from gptq_qqq_calibration_gb300 import Int8Linear, Rows8
    d, f = 64, 72
    _, (wq, ws), _ = make(1, d, f, torch.bfloat16, 1)
    op = Int8Linear(d, f, tokens=4, train_tokens=4)
    none = Rows8(torch.empty((0, d), dtype=torch.int8, device="cuda"), torch.empty(0, device="cuda"))
    assert op.forward(torch.empty((0, d), dtype=torch.bfloat16, device="cuda"), rows8(wq, ws)).shape == (0, f)
    dx, dw = op.backward(torch.empty((0, f), dtype=torch.bfloat16, device="cuda"), none, rows8(wq, ws))
    assert dx.shape == (0, d) and dw.shape == (f, d) and not dw.any()
    op.sync()


def test_rows_behind_the_last_token_are_left():
    from gptq_qqq_calibration_gb300 import Int8Linear
    d, f = 272, 264
    for n in (3, 50, 200):
        x, (wq, ws), _ = make(n, d, f, torch.float16, n)
        out = torch.full((n + 20, f), 9.0, dtype=torch.float16, device="cuda")
        op = Int8Linear(d, f, tokens=n, dtype=torch.float16)
        op.forward(x.cuda(), rows8(wq, ws), out=out[:n])
        op.sync()
        assert (out[n:] == 9.0).all() and same(out[:n], product(*formula(x, 0), wq, ws, torch.float16))


def test_rows_past_32_bit_offsets():
    """More than 2^32 elements of y."""
    from gptq_qqq_calibration_gb300 import Int8Linear
    n, d, f = 400000, 64, 11008
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn((n, d), generator=g, device="cuda").bfloat16()
    _, (wq, ws), _ = make(1, d, f, torch.bfloat16, 40)
    op = Int8Linear(d, f, tokens=n)
    y = op.forward(X, rows8(wq, ws))
    op.sync()
    at = [0, 195000, 195083, 195084, 390168, n - 1]
    assert same(y[at], product(*formula(X[at].cpu(), 0), wq, ws, torch.bfloat16))


def test_leading_shapes_and_repeatability():
    from gptq_qqq_calibration_gb300 import Int8Linear
    n, d, f = 60, 528, 264
    x, (wq, ws), dy = make(n, d, f, torch.bfloat16, 4)
    op = Int8Linear(d, f, tokens=n, train_tokens=n)
    w = rows8(wq, ws)
    y = op.forward(x.cuda().view(3, 20, d), w)
    assert y.shape == (3, 20, f) and torch.equal(y.view(n, f), op.forward(x.cuda(), w))
    rows = rows8(*formula(x, 0))
    first = op.backward(dy.cuda(), rows, w)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, op.backward(dy.cuda(), rows, w)))
    op.sync()


def test_streams_share_one_workspace():
    from gptq_qqq_calibration_gb300 import Int8Linear
    d, f = 2064, 1400
    sets = []
    for k, n in enumerate((5, 40, 300, 300)):
        x, (wq, ws), dy = make(n, d, f, torch.bfloat16, 20 + k)
        sets.append((x.cuda(), rows8(*formula(x, 0)), rows8(wq, ws), dy.cuda()))
    op = Int8Linear(d, f, tokens=300, train_tokens=300)
    want = [(op.forward(x, w), *op.backward(dy, r, w)) for x, r, w, dy in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        got = [(op.forward(x, w, stream=s), *op.backward(dy, r, w, stream=s))
               for (x, r, w, dy), s in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    op.sync()


@pytest.mark.parametrize("n", [4, 100])
def test_graph_capture(n):
    from gptq_qqq_calibration_gb300 import Int8Linear
    d, f = 528, 1400
    x, (wq, ws), dy = make(n, d, f, torch.bfloat16, 30)
    op = Int8Linear(d, f, tokens=n, train_tokens=n)
    X, w, rows, DY = x.cuda(), rows8(wq, ws), rows8(*formula(x, 0)), dy.cuda()
    want = (op.forward(X, w), *op.backward(DY, rows, w))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (op.forward(X, w), *op.backward(DY, rows, w))
    other = torch.cuda.Stream()
    late = op.forward(X, w, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(late, want[0])
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    op.sync()


def test_weights_written_just_before():
    """The weights of a call may be the result of the kernel before it on the stream."""
    from gptq_qqq_calibration_gb300 import Int8Linear, quantize_rows
    n, d, f = 64, 4096, 4096
    x, _, _ = make(n, d, 8, torch.bfloat16, 3)
    X = x.cuda()
    op = Int8Linear(d, f, tokens=n)
    g = torch.Generator(device="cuda").manual_seed(3)
    masters = [torch.randn((f, d), generator=g, device="cuda") for _ in range(4)]
    want = []
    for m in masters:
        w = quantize_rows(m)
        torch.cuda.synchronize()
        want.append(op.forward(X, w))
        torch.cuda.synchronize()
    from gptq_qqq_calibration_gb300 import Rows8
    from gptq_qqq_calibration_gb300.rows8 import rows8_quantize
    codes, scale = torch.empty((f, d), dtype=torch.int8, device="cuda"), torch.empty(f, device="cuda")
    got = []
    for _ in range(3):
        for m in masters:
            rows8_quantize(m, 0, codes, scale)
            got.append(op.forward(X, Rows8(codes, scale)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[k % 4]) for k, a in enumerate(got))
    op.sync()


@pytest.mark.parametrize("n", [40, 100, 300])  # a tile width of each kernel
@pytest.mark.parametrize("limit", [0, 500, 2000, 8000])
def test_waits_that_run_out_end_the_kernel(limit, n):
    """Split tiles with a limit that some waits keep and others do not: the kernel ends,
    says so, and the handle works again.  (Sums over enough columns that a tile's end is
    waited for longer than one attempt of a wait lasts.)"""
    from gptq_qqq_calibration_gb300 import HessError, Int8Linear
    from gptq_qqq_calibration_gb300.int8_linear import int8_linear_set_timeout
    d, f = 16400, 4096
    x, (wq, ws), _ = make(n, d, f, torch.bfloat16, 60)
    op = Int8Linear(d, f, tokens=n)
    X, w = x.cuda(), rows8(wq, ws)
    want = op.forward(X, w)
    op.sync()
    timeouts = 0
    for _ in range(6):
        int8_linear_set_timeout(op.handle, limit)
        op.forward(X, w)
        int8_linear_set_timeout(op.handle, 2_000_000_000)
        try:
            op.sync()
        except HessError as e:
            assert "TIMEOUT" in str(e)
            timeouts += 1
        assert torch.equal(op.forward(X, w), want)
    assert timeouts > 0 or limit > 0
    op.sync()


def test_two_threads_share_a_handle():
    """Host threads with streams of their own: calls of every kernel, forward and backward."""
    import threading
    from gptq_qqq_calibration_gb300 import Int8Linear, quantize_rows
    d, f = 1040, 2056
    op = Int8Linear(d, f, tokens=300, train_tokens=300)
    work = []
    for k, n in enumerate((1, 2, 9, 30, 70, 300)):
        x, (wq, ws), dy = make(n, d, f, torch.bfloat16, 70 + k)
        X, w = x.cuda(), rows8(wq, ws)
        rows = quantize_rows(X)
        work.append((X, w, rows, dy.cuda()))
    want = [(op.forward(X, w), *op.backward(dy, rows, w)) for X, w, rows, dy in work]
    torch.cuda.synchronize()
    wrong = []

    def run(order):
        stream = torch.cuda.Stream()
        for k in order:
            X, w, rows, dy = work[k]
            got = (op.forward(X, w, stream=stream), *op.backward(dy, rows, w, stream=stream))
            stream.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                wrong.append(k)

    threads = [threading.Thread(target=run, args=(order * 10,)) for order in ([0, 1, 2, 3, 4, 5], [5, 3, 1, 4, 2, 0])]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    op.sync()


def test_autograd_node():
    from gptq_qqq_calibration_gb300 import Int8Linear, quantize_rows
    n, d, f = 40, 272, 136
    g = torch.Generator().manual_seed(8)
    X = torch.randn((2, n // 2, d), generator=g).bfloat16().cuda().requires_grad_()
    W = (torch.randn((f, d), generator=g) / 16).bfloat16().cuda().requires_grad_()
    op = Int8Linear(d, f, tokens=n, train_tokens=n)
    y = op(X, W)
    dy = torch.randn((2, n // 2, f), generator=g).bfloat16().cuda()
    y.backward(dy)
    rows, w = quantize_rows(X.detach()), quantize_rows(W.detach())
    assert torch.equal(y, op.forward(X.detach(), w))
    dx, dw = op.backward(dy, rows, w)
    assert torch.equal(X.grad, dx) and torch.equal(W.grad, dw)
    # one of the two, and a gradient that is not laid out in order
    X2 = X.detach().requires_grad_()
    big = torch.zeros((2, f, n // 2 + 1), dtype=torch.bfloat16, device="cuda")
    big[:, :, 1:] = dy.transpose(1, 2)
    op(X2, W.detach()).backward(big[:, :, 1:].transpose(1, 2))
    assert torch.equal(X2.grad, dx)
    # no tokens at all
    W2 = W.detach().requires_grad_()
    none = torch.zeros((0, d), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    op(none, W2).backward(torch.zeros((0, f), dtype=torch.bfloat16, device="cuda"))
    assert none.grad.shape == (0, d) and (W2.grad == 0).all()
    op.sync()


def test_refusals():
    from gptq_qqq_calibration_gb300 import HessError, Int8Linear, Rows8, _lib
    n, d, f = 16, 64, 128
    x, (wq, ws), dy = make(n, d, f, torch.bfloat16, 1)
    X, w, DY, rows = x.cuda(), rows8(wq, ws), dy.cuda(), rows8(*formula(x, 0))
    grouped = rows8(*formula(x, 32), 32)
    op = Int8Linear(d, f, tokens=n, train_tokens=8)
    for bad in (lambda: op.forward(x, w), lambda: op.forward(X.half(), w), lambda: op.forward(X[:, :32], w),
                lambda: op.forward(X, Rows8(w.codes[:64], w.scale)), lambda: op.forward(X, Rows8(w.codes, w.scale[:9])),
                lambda: op.forward(X, w._replace(group=32)), lambda: op.forward(grouped, w),
                lambda: op.forward(X, w, out=torch.empty((3, f), dtype=torch.bfloat16, device="cuda")),
                lambda: op.backward(DY[:3], rows, w), lambda: op.backward(DY, grouped._replace(group=64), w),
                lambda: Int8Linear(d, f, 4, dtype=torch.float64)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: Int8Linear(72, f, 4), lambda: Int8Linear(d, 129, 4), lambda: Int8Linear(65552, f, 4),
                lambda: Int8Linear(d, f, -1), lambda: Int8Linear(d, f, 4, dtype=torch.float32),
                lambda: op.backward(DY, rows, w),  # 16 tokens, workspace for 8
                lambda: Int8Linear(d, f, tokens=8).forward(X, w)):
        with pytest.raises(HessError):
            bad()
    lib = _lib.load()
    out = torch.empty((n, f), dtype=torch.bfloat16, device="cuda")
    hostbuf = torch.zeros(n * f, dtype=torch.bfloat16).data_ptr()
    args = [op.handle, X.data_ptr(), n, w.codes.data_ptr(), w.scale.data_ptr(), out.data_ptr(), None]
    for at, wrong in ((0, None), (1, None), (1, hostbuf), (1, X.data_ptr() + 2), (2, -1), (2, 17), (3, None),
                      (3, hostbuf), (3, w.codes.data_ptr() + 8), (4, None), (4, w.scale.data_ptr() + 2), (5, None),
                      (5, hostbuf), (5, out.data_ptr() + 2), (5, X.data_ptr()), (5, w.codes.data_ptr() + 64),
                      (5, w.scale.data_ptr())):
        bad = list(args)
        bad[at] = wrong
        assert lib.int8_linear_forward(*bad) == _lib.HESS_ERR_INVALID, (at, wrong)
    assert lib.int8_linear_forward(*args) == _lib.HESS_OK
    args = [op.handle, rows.codes.data_ptr(), rows.scale.data_ptr(), n, w.codes.data_ptr(), w.scale.data_ptr(),
            out.data_ptr(), None]
    for at, wrong in ((1, None), (1, rows.codes.data_ptr() + 8), (2, None), (2, hostbuf), (6, rows.codes.data_ptr()),
                      (6, rows.scale.data_ptr())):
        bad = list(args)
        bad[at] = wrong
        assert lib.int8_linear_forward_rows8(*bad) == _lib.HESS_ERR_INVALID, (at, wrong)
    dx = torch.empty((8, d), dtype=torch.bfloat16, device="cuda")
    dw = torch.empty((f, d), dtype=torch.bfloat16, device="cuda")
    args = [op.handle, DY.data_ptr(), 8, rows.codes.data_ptr(), rows.scale.data_ptr(), 0, w.codes.data_ptr(),
            w.scale.data_ptr(), dx.data_ptr(), dw.data_ptr(), None]
    for at, wrong in ((0, None), (1, None), (1, hostbuf), (1, DY.data_ptr() + 2), (2, 9), (2, -1), (3, None),
                      (4, None), (6, None), (7, None), (8, DY.data_ptr()), (8, dw.data_ptr()), (8, rows.codes.data_ptr()),
                      (9, w.codes.data_ptr()), (9, dx.data_ptr()), (9, hostbuf)):
        bad = list(args)
        bad[at] = wrong
        assert lib.int8_linear_backward(*bad) == _lib.HESS_ERR_INVALID, (at, wrong)
    bad = list(args)
    bad[5] = 48
    assert lib.int8_linear_backward(*bad) == _lib.HESS_ERR_UNSUPPORTED
    for leave in ((6, 7, 8), (3, 4, 9)):  # what an unwanted result alone needs may be missing
        some = list(args)
        for at in leave:
            some[at] = None
        assert lib.int8_linear_backward(*some) == _lib.HESS_OK
    op.sync()
