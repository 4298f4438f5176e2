"""Codes of rows whose scale is about float32's smallest normal number.

The scale's own rounding is then a step of 2^-149 as well, and the remainder x - (m + 1/2) s, whose
sign decides a code, can be half of such a step: 2^-150, which float32 does not hold.  Values are
taken on both sides of every half, and compared with the formula in 64 bits, bit for bit (quotients of
two float32 numbers are a half or 2^-25 of themselves away from one).
"""

import pytest
import torch

from test_gpu_int8_linear import product, rows8, same
from test_gpu_rows8 import check, formula

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


def near_halves_f32(n=24, seed=1):
    """[n, 1024]: a maximum, and float32 values beside (m + 1/2) s for every m, of rows whose scales
    lie in [2^-128, 2^-123] and whose maxima have every kind of remainder by 127."""
    g = torch.Generator().manual_seed(seed)
    step = 2.0 ** -149
    rows = []
    for k in range(n):
        low = 2.0 ** (-128 + k % 6)
        a = round((1.0 + torch.rand((), generator=g).item()) * 127 * low / step) * step
        top = torch.tensor(a, dtype=torch.float64).float()
        s = (top.double() / 127).float().double()
        half = (torch.arange(127, dtype=torch.float64) + 0.5) * s
        at = half.float()
        around = [at, torch.nextafter(at, torch.tensor(0.0)), torch.nextafter(at, torch.tensor(1.0)),
                  torch.nextafter(torch.nextafter(at, torch.tensor(0.0)), torch.tensor(0.0))]
        x = torch.cat(around + [-v for v in around])
        x = torch.cat([x[x.abs() <= top], top[None]])
        rows.append(torch.nn.functional.pad(x, (0, 1024 - x.numel())))
    return torch.stack(rows)


def halves_bf16():
    """[n, 256] bf16: every maximum whose scale lies in [2^-127, 2^-124], its half (63.5 scales,
    up to the scale's rounding) and the numbers below it."""
    rows = []
    for e in (-128, -127, -126, -125, -124, -123):
        for k in range(128, 256):
            top = k * 2.0 ** e
            below = torch.arange(1, 256, dtype=torch.float64) * (top / 256)
            x = torch.cat([torch.tensor([top, top / 2, -top / 2, 111 * 2.0 ** e], dtype=torch.float64), below])[:256]
            rows.append(x.clamp(-top, top))
    return torch.stack(rows).to(torch.bfloat16)


def test_the_row_that_shows_it():
    """Maximum 222 2^-126 and x = 111 2^-126: s = 14663551 2^-149, x / s = 63.49999997."""
    from gptq_qqq_calibration_gb300 import quantize_rows
    x = torch.zeros((2, 16), dtype=torch.bfloat16)
    x[:, 0], x[:, 1], x[:, 2] = 222 * 2.0 ** -126, 111 * 2.0 ** -126, -111 * 2.0 ** -126
    rows = quantize_rows(x.cuda())
    assert rows.codes[0, :3].tolist() == [127, 63, -63]
    assert rows.scale[0].item() == 14663551 * 2.0 ** -149


@pytest.mark.parametrize("width", [1024, 1023, 256])
@pytest.mark.parametrize("group", [0, 32, 128])
def test_float32_rows(width, group):
    check(near_halves_f32()[:, -width:].contiguous(), group)


@pytest.mark.parametrize("group", [0, 64])
def test_bf16_rows(group):
    x = halves_bf16()
    check(x, group)
    check(torch.cat([x, torch.zeros((x.shape[0], 1024), dtype=x.dtype)], 1), group)  # long rows, many
    check(torch.cat([x, torch.zeros((x.shape[0], 1791), dtype=x.dtype)], 1)[:100].contiguous(), group)  # odd ones


@pytest.mark.parametrize("n", [1, 2, 3, 16, 40])
def test_tokens_of_the_integer_layer(n):
    """Every kernel of the layer quantizes its tokens alike.  The weight's scales bring the results
    back into the type's range."""
    from gptq_qqq_calibration_gb300 import Int8Linear
    x = halves_bf16()
    x = x[(x.float().abs().amax(dim=1) >= 127 * 2.0 ** -126)]  # normal scales
    d, f = 256, 264
    g = torch.Generator().manual_seed(n)
    wq = torch.randint(-127, 128, (f, d), generator=g).to(torch.int8)
    ws = torch.full((f,), 2.0 ** 120)
    op = Int8Linear(d, f, tokens=n)
    w = rows8(wq, ws)
    for first in range(0, x.shape[0] - n, max(n, x.shape[0] // 60)):
        t = x[first:first + n]
        assert same(op.forward(t.cuda(), w), product(*formula(t, 0), wq, ws, torch.bfloat16)), first
    op.sync()
    op.close()
