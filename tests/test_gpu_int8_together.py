"""A run of the 8-bit operators together, as a quantized block is calibrated, tuned
and served: the projections' output is calibrated on, GPTQ's codes become the integer
layer's weight, the step's activations are kept in 8 bits, and the same layer then
runs token by token.

Values are followed from one operator to the next in 64 bits, each step from what
the GPU handed to it, so that an operator's own tolerance holds at every step (the
integer layer's forward: none)."""

import pytest
import torch

from test_gpu_gated_ff import check, reference
from test_gpu_int8_linear import check as check_sum, product
from test_gpu_rows8 import formula, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def inputs(tokens, d, f, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x, dy = torch.randn((tokens, d), generator=g), 0.1 * torch.randn((tokens, d), generator=g)
    gate, up = (torch.randn((f, d), generator=g) / d ** 0.5 for _ in range(2))
    down = torch.randn((d, f), generator=g) / f ** 0.5
    return [t.to(dtype).cuda() for t in (x, gate, up, down, dy)]


def quantized_down(h, down):
    from gptq_qqq_calibration_gb300 import GPTQ, Hessian, Rows8
    hessian = Hessian(h.shape[1])
    hessian.add_batch(h)
    gptq = GPTQ(h.shape[1], down.shape[0])
    gptq.prepare(hessian, 0.01)
    q = gptq.quantize(down, group_size=-1)
    # the codes and scales stand for the quantized weight, bit for bit
    assert torch.equal(q["codes"].float() * q["scales"].view(-1, 1), q["Wq"])
    return Rows8(q["codes"], q["scales"])


@pytest.mark.parametrize("tokens", [201, 640])
def test_calibrated_tuned_and_served(tokens):
    from gptq_qqq_calibration_gb300 import GatedFF, Int8Linear, quantize_rows, restore_rows
    d, f, dtype = 256, 640, torch.bfloat16
    x, gate, up, down, dy = inputs(tokens, d, f, dtype, tokens)
    block = GatedFF(d, f, train_tokens=tokens, rows8=True)
    layer = Int8Linear(f, d, tokens=tokens, train_tokens=tokens)
    h = block.forward(x, gate, up)
    weight = quantized_down(h, down)
    wq, ws = weight.codes.cpu(), weight.scale.cpu().view(-1)

    # the step: h as 8-bit rows, x as an 8-bit checkpoint
    rows, kept = quantize_rows(h), quantize_rows(x, group=128)
    y = layer.forward(rows, weight)
    hq, hs = formula(h.cpu(), 0)
    assert torch.equal(rows.codes.cpu(), hq) and torch.equal(rows.scale.cpu(), hs)
    assert torch.equal(y.cpu(), product(hq, hs, wq, ws, dtype))
    dh, dw = layer.backward(dy, rows, weight)
    for t, a, b in ((dh, dy.cpu(), values(wq, ws, 0, dtype)), (dw, dy.cpu().T, values(hq, hs, 0, dtype))):
        a, b = a.double(), b.double()
        check_sum(t, a @ b, (a.shape[1] / 16 + 8) * 2.0 ** -23 * (a.abs() @ b.abs()), dtype)
    got = block.backward(kept, gate, up, dh)
    ref = reference(restore_rows(kept, dtype).cpu(), gate.cpu(), up.cpu(), dh.cpu(), "silu")
    for t, k in zip(got, ("dx", "dwg", "dwu")):
        check(t, ref[k], dtype)

    # the same two layers for requests of every size: the integer layer gives each token the
    # bits that it has in the batch
    for t0, n in ((0, 1), (1, 2), (3, 3), (6, 16), (22, 17), (39, 100)):
        part = h[t0:t0 + n]
        assert torch.equal(layer.forward(part, weight), y[t0:t0 + n]), n
        assert torch.equal(layer.forward(quantize_rows(part), weight), y[t0:t0 + n]), n
    block.sync()
    layer.sync()


def test_the_step_as_a_graph():
    """The whole step captured once and replayed on other values: its operators follow
    each other on one stream, and each reads what the one before wrote."""
    from gptq_qqq_calibration_gb300 import GatedFF, Int8Linear, quantize_rows
    tokens, d, f, dtype = 301, 192, 384, torch.float16
    sets = [inputs(tokens, d, f, dtype, 50 + k) for k in range(3)]
    block = GatedFF(d, f, train_tokens=tokens, dtype=dtype, rows8=True)
    layer = Int8Linear(f, d, tokens=tokens, train_tokens=tokens, dtype=dtype)
    weight = quantize_rows(sets[0][3])

    def step(x, gate, up, dy):
        kept = quantize_rows(x, group=128)
        rows = quantize_rows(block.forward(x, gate, up))
        y = layer.forward(rows, weight)
        dh, dw = layer.backward(dy, rows, weight)
        return (y, dw, *block.backward(kept, gate, up, dh))

    want = [[t.clone() for t in step(s[0], s[1], s[2], s[4])] for s in sets]
    given = [sets[0][i].clone() for i in (0, 1, 2, 4)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*given)
    for s, w in ((sets[1], want[1]), (sets[2], want[2]), (sets[0], want[0])):
        for t, i in zip(given, (0, 1, 2, 4)):
            t.copy_(s[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, w))
    block.sync()
    layer.sync()


def test_nodes_of_one_autograd_graph():
    """The operators' nodes behind one another, eager and captured (the backward pass with
    its forward pass, on leaves of its own), against the calls one by one."""
    from gptq_qqq_calibration_gb300 import GatedFF, Int8Linear, quantize_rows
    tokens, d, f = 150, 128, 256
    x, gate, up, down, dy = inputs(tokens, d, f, torch.bfloat16, 9)
    block = GatedFF(d, f, train_tokens=tokens, rows8=True)
    layer = Int8Linear(f, d, tokens=tokens, train_tokens=tokens)
    rows, weight = quantize_rows(block.forward(x, gate, up)), quantize_rows(down.float())
    y = layer.forward(rows, weight)
    dh, dw = layer.backward(dy, rows, weight)
    want = (*block.backward(quantize_rows(x, group=128), gate, up, dh), dw.float())

    def leaves():
        return [t.clone().requires_grad_() for t in (x, gate, up, down.float())]  # an fp32 master among them

    def run(a):
        out = layer(block(*a[:3]), a[3])
        return out, torch.autograd.grad(out, a, dy)

    out, got = run(leaves())
    assert torch.equal(out, y) and all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.no_grad():  # nothing is kept, and nothing changes
        assert torch.equal(layer(block(x, gate, up), down), y)
    del out, got
    own = leaves()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, got = run(own)
    for t in (out, *got):
        t.detach().zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, y) and all(torch.equal(a, b) for a, b in zip(got, want))
    block.sync()
    layer.sync()
