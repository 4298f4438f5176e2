"""Feed-forward gradients from an 8-bit checkpoint of the input.

Bit for bit those of the call on the restored values, which test_gpu_rows8.py and
test_gpu_gated_ff.py hold to their formulas."""

import pytest
import torch

from test_gpu_gated_ff import check, make, reference
from test_gpu_rows8 import formula, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("dtype,kind", [(torch.bfloat16, "silu"), (torch.float16, "gelu_tanh")])
@pytest.mark.parametrize("n,d,f,group", [(1, 8, 8, 0), (1, 64, 128, 32), (17, 520, 1400, 128), (129, 64, 72, 0),
                                         (300, 264, 136, 64), (600, 1024, 640, 256)])
def test_same_bits_as_the_restored_values(n, d, f, group, dtype, kind):
    from gptq_qqq_calibration_gb300 import GatedFF, Rows8, quantize_rows, restore_rows
    x, wg, wu, dh = make(n, d, f, dtype, n + d)
    G, U, D = wg.cuda(), wu.cuda(), dh.cuda()
    op = GatedFF(d, f, train_tokens=n, dtype=dtype, activation=kind, rows8=True)
    rows = quantize_rows(x.cuda(), group=group)
    want = op.backward(restore_rows(rows, dtype), G, U, D)
    got = op.backward(rows, G, U, D)
    assert same(want, got)
    ref = reference(values(*formula(x, group), group, dtype), wg, wu, dh, kind)
    for t, k in zip(got, ("dx", "dwg", "dwu")):
        check(t, ref[k], dtype)
    # codes that start anywhere, and one result without the other
    flat = torch.empty(n * d + 3, dtype=torch.int8, device="cuda")
    flat[3:] = rows.codes.view(-1)
    moved = Rows8(flat[3:].view(n, d), rows.scale, group)
    assert same(op.backward(moved, G, U, D), want)
    assert torch.equal(op.backward(rows, G, U, D, want_dw=False)[0], want[0])
    assert same(op.backward(rows, G, U, D, want_dx=False)[1:], want[1:])
    op.sync()


def test_autograd_node_keeps_8_bit_rows():
    from gptq_qqq_calibration_gb300 import GatedFF, quantize_rows
    n, d, f = 48, 256, 384
    x, wg, wu, dh = make(n, d, f, torch.bfloat16, 3)
    X, G, U = (t.cuda().requires_grad_() for t in (x, wg, wu))
    op = GatedFF(d, f, train_tokens=n, rows8=True)
    sizes = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: (sizes.append((t.dtype, t.numel())), t)[1], lambda t: t):
        h = op(X, G, U)
    assert (torch.bfloat16, n * d) not in sizes and (torch.int8, n * d) in sizes
    assert torch.equal(h, op.forward(x.cuda(), wg.cuda(), wu.cuda()))
    h.backward(dh.cuda())
    want = op.backward(quantize_rows(x.cuda(), group=128), wg.cuda(), wu.cuda(), dh.cuda())
    assert same((X.grad, G.grad, U.grad), want)
    op.sync()


def test_streams_and_graphs():
    from gptq_qqq_calibration_gb300 import GatedFF, quantize_rows
    n, d, f = 700, 512, 1024
    op = GatedFF(d, f, train_tokens=n, rows8=True)
    sets = []
    for k in range(3):
        x, wg, wu, dh = (t.cuda() for t in make(n, d, f, torch.bfloat16, 20 + k))
        sets.append((quantize_rows(x, group=128), wg, wu, dh))
    want = [op.backward(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = [op.backward(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = op.backward(*sets[1])
    op.backward(*sets[0])
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, want[1])
    op.sync()


def test_refusals():
    from gptq_qqq_calibration_gb300 import GatedFF, HessError, Rows8, _lib, quantize_rows
    n, d, f = 16, 64, 128
    x, wg, wu, dh = (t.cuda() for t in make(n, d, f, torch.bfloat16, 1))
    rows = quantize_rows(x)
    with pytest.raises(HessError, match="reserve"):
        GatedFF(d, f, train_tokens=n).backward(rows, wg, wu, dh)
    with pytest.raises(HessError):
        GatedFF(d, f, rows8=True)  # no train_tokens
    op = GatedFF(d, f, train_tokens=n, rows8=True)
    for bad in (rows._replace(group=32), rows._replace(scale=rows.scale[:3]), rows._replace(codes=rows.codes.short()),
                Rows8(rows.codes[:, :32], rows.scale)):
        with pytest.raises(ValueError):
            op.backward(bad, wg, wu, dh)
    lib = _lib.load()
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    hostbuf = torch.zeros(n * f, dtype=torch.bfloat16).data_ptr()
    args = [op.handle, rows.codes.data_ptr(), rows.scale.data_ptr(), 0, n, wg.data_ptr(), wu.data_ptr(),
            dh.data_ptr(), dx.data_ptr(), dwg.data_ptr(), dwu.data_ptr(), None]
    for at, wrong in ((0, None), (1, None), (1, hostbuf), (2, None), (2, hostbuf), (2, rows.scale.data_ptr() + 2),
                      (4, 17), (4, -1), (5, None), (7, hostbuf), (8, rows.codes.data_ptr()), (9, rows.scale.data_ptr()),
                      (10, None)):
        bad = list(args)
        bad[at] = wrong
        assert lib.gated_ff_backward_rows8(*bad) == _lib.HESS_ERR_INVALID, (at, wrong)
    bad = list(args)
    bad[3] = 16
    assert lib.gated_ff_backward_rows8(*bad) == _lib.HESS_ERR_UNSUPPORTED
    assert lib.gated_ff_backward_rows8(*args) == _lib.HESS_OK
    op.sync()
