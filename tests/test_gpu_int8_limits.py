"""The integer layer's waits with a limit: a call whose waits all kept it is right, any other says so.

Limits are spread over the time that a call takes, so that waits of every role run out at
some of them; the kernel always ends, and the handle works again.
"""

import pytest
import torch

from test_gpu_int8_linear import make, product, rows8
from test_gpu_rows8 import formula

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()


# tokens of every tile width; weight rows that leave a converter warp partly or wholly idle
@pytest.mark.parametrize("n,d,f", [(33, 4096, 1400), (40, 16400, 4096), (100, 4096, 4096), (300, 4096, 2056)])
def test_no_wrong_result_without_a_word(n, d, f):
    from gptq_qqq_calibration_gb300 import HessError, Int8Linear
    from gptq_qqq_calibration_gb300.int8_linear import int8_linear_set_timeout
    x, (wq, ws), _ = make(n, d, f, torch.bfloat16, n)
    want = product(*formula(x, 0), wq, ws, torch.bfloat16).cuda()
    op = Int8Linear(d, f, tokens=n)
    X, w = x.cuda(), rows8(wq, ws)
    assert torch.equal(op.forward(X, w), want)
    op.sync()
    ended = 0
    for limit in (0, 100, 200, 400, 700, 1000, 1500, 2000, 3000, 4000, 6000, 9000, 14000, 20000):
        for _ in range(3):
            out = torch.full_like(want, float("nan"))
            int8_linear_set_timeout(op.handle, limit)
            op.forward(X, w, out=out)
            int8_linear_set_timeout(op.handle, 2_000_000_000)
            try:
                op.sync()
            except HessError as e:
                assert "TIMEOUT" in str(e)
                ended += 1
            else:
                assert torch.equal(out, want), limit
    # (one attempt of a wait lasts longer than any wait of the narrower layers)
    assert ended > 0 or d < 16400
    assert torch.equal(op.forward(X, w), want)
    op.sync()
    op.close()
