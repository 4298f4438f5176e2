"""The scale a / 127 is the correctly rounded quotient, for every significand of a.

64 bits hold the quotient to 2^-53 of itself, and no quotient by 127 that is not a float32 number or
halfway between two lies nearer to a halfway point than 2^-25 / 127 of itself: so the 64-bit quotient
rounds to the same float32 number as the exact one."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


# the fast form's range begins at 2^-100; below it the scale is divided, and from 2^-119 on subnormal
@pytest.mark.parametrize("exponent", [0, 127 - 1, -100, -101, -119, -126])
def test_every_significand(exponent):
    from gptq_qqq_calibration_gb300 import quantize_rows
    bits = torch.arange(1 << 23, dtype=torch.int32, device="cuda") + ((exponent + 127) << 23)
    a = bits.view(torch.float32)
    rows = quantize_rows(-a[:, None])  # a value is a row of its own
    assert torch.equal(rows.scale, (a.double() / 127).float())
    assert bool((rows.codes == -127).all()) or exponent < -100


def test_every_subnormal_maximum():
    from gptq_qqq_calibration_gb300 import quantize_rows
    a = torch.arange(1 << 23, dtype=torch.int32, device="cuda").view(torch.float32)
    rows = quantize_rows(a[:, None])
    s = (a.double() / 127).float()
    assert torch.equal(rows.scale, s)
    q = torch.where(s > 0, torch.round(a.double() / s.double()).clamp(-127, 127), torch.zeros_like(a).double())
    assert torch.equal(rows.codes[:, 0], q.to(torch.int8))
