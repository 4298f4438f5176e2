"""The example that runs calibration, quantization, the distillation loss and
the feed-forward gradients together."""

import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recover_block.py")


def test_recovery_lowers_the_loss():
    from gptq_qqq_calibration_gb300 import build as b
    b.build()
    spec = importlib.util.spec_from_file_location("recover_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.run(d=256, f=512, vocab=1003, tokens=700, steps=15)
    assert r["quantized"] > 0 and r["recovered"] < 0.9 * r["quantized"]
    # one token at a time the sums are taken in another order: bf16 logits may round differently
    assert abs(r["token_by_token"] - r["same_tokens"]) <= 0.05 * (r["same_tokens"] + 0.01)
