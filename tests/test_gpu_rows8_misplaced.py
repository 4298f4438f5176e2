"""8-bit rows where a call takes a tensor, and tensors where it takes 8-bit rows: refused by name."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def tensors(n, d, f):
    g = torch.Generator().manual_seed(1)
    return [torch.randn(s, generator=g).bfloat16().cuda() for s in ((n, d), (f, d), (f, d), (n, f))]


@pytest.mark.parametrize("rows8", [False, True])
@pytest.mark.parametrize("n", [4, 200])
def test_feed_forward(n, rows8):
    from gptq_qqq_calibration_gb300 import GatedFF, quantize_rows
    x, wg, wu, dh = tensors(n, 64, 128)
    op = GatedFF(64, 128, train_tokens=n, rows8=rows8)
    rows = quantize_rows(x)
    for call in (op.forward, op):
        with pytest.raises(ValueError, match="8-bit rows"):
            call(rows, wg, wu)
        with torch.no_grad(), pytest.raises(ValueError, match="8-bit rows"):
            call(rows, wg, wu)
    with pytest.raises(ValueError, match="8-bit rows"):
        op.forward(rows, wg, wu, out=torch.empty_like(dh))
    assert torch.equal(op.forward(x, wg, wu), op(x, wg, wu))
    op.sync()


def test_integer_layer_and_rows():
    from gptq_qqq_calibration_gb300 import Int8Linear, quantize_rows, restore_rows
    n, d, f = 4, 64, 128
    x, w, _, dy = tensors(n, d, f)
    op = Int8Linear(d, f, tokens=n, train_tokens=n)
    rows, weight = quantize_rows(x), quantize_rows(w)
    with pytest.raises(ValueError, match="tensor"):
        op(rows, w)
    with pytest.raises(ValueError, match="tensor"):
        op(x, weight)
    with pytest.raises(ValueError, match="tensor"):
        quantize_rows(rows)
    for bad in (w, weight.codes, (weight.codes, weight.scale)):
        with pytest.raises(ValueError, match="weight must be 8-bit rows"):
            op.forward(x, bad)
        with pytest.raises(ValueError, match="weight must be 8-bit rows"):
            op.backward(dy, rows, bad)
    for bad in (x, rows.codes):
        with pytest.raises(ValueError, match="X must be 8-bit rows"):
            op.backward(dy, bad, weight)
        with pytest.raises(ValueError, match="rows must be 8-bit rows"):
            restore_rows(bad)
    op.forward(rows, weight)
    op.sync()
