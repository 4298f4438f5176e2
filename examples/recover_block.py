"""Calibrate, quantize and recover one feed-forward block against its original.

The original ("teacher") block is y = x + W_down h, h = silu(W_gate x) * (W_up x),
followed by an output head.  The quantized block runs its down projection as it is
served: in 8-bit integers, on h quantized per token.  The example

  1. runs the gated projections over calibration tokens (``GatedFF``) and
     collects the Hessian of h, the down projection's input (``Hessian``);
  2. quantizes W_down with it (``GPTQ``), whose codes and scales are the weight of
     the integer layer (``Int8Linear``);
  3. keeps the teacher's top logits and its log-sum per token, and scores the
     quantized block against them (``distill_forward``);
  4. tunes W_gate and W_up with the quantized W_down in place: the gradient of
     the distillation loss (``distill_step``) goes back through the head, through
     the integer layer (``Int8Linear.backward``, straight through the rounding of
     h) and through the projections (``GatedFF.backward``), which read x from an
     8-bit checkpoint (``quantize_rows``);
  5. scores one token at a time, as a server would run it.

    python examples/recover_block.py [--d 512 --f 1408 --vocab 4000 --tokens 2048 --steps 30]

d is a multiple of 8, f of 16.
"""

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from gptq_qqq_calibration_gb300 import (GPTQ, GatedFF, Hessian, Int8Linear, Rows8, distill_forward,  # noqa: E402
                                        distill_step, quantize_rows)


def run(d=512, f=1408, vocab=4000, tokens=2048, steps=30, top=64, temperature=1.0, lr=0.05, seed=0):
    """Returns the mean losses {"quantized", "recovered", "token_by_token"}."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale):
        return (scale * torch.randn(shape, generator=gen, device="cuda")).bfloat16()

    w_gate, w_up = normal(f, d, scale=d ** -0.5), normal(f, d, scale=d ** -0.5)
    w_down, w_head = normal(d, f, scale=2.0 * f ** -0.5), normal(vocab, d, scale=2.0 * d ** -0.5)
    x = normal(tokens, d, scale=1.0)
    block = GatedFF(d, f, train_tokens=tokens, rows8=True)
    down = Int8Linear(f, d, tokens=tokens, train_tokens=tokens)

    # 1. the down projection's input and its Hessian, in ragged batches
    hessian = Hessian(f)
    for part in x.split(tokens // 3 + 1):
        hessian.add_batch(block.forward(part, w_gate, w_up))

    # 2. the quantized down projection
    gptq = GPTQ(f, d)
    gptq.prepare(hessian, 0.01)
    quantized = gptq.quantize(w_down, group_size=-1)
    w_q = Rows8(quantized["codes"], quantized["scales"])

    # 3. the teacher's top logits, and the quantized block against them
    teacher = ((x + block.forward(x, w_gate, w_up) @ w_down.t()) @ w_head.t()).float()
    top_logits, top_index = torch.topk(teacher, top, dim=1)
    lists = dict(top_logits=top_logits, top_index=top_index.int(), temperature=temperature,
                 teacher_lse=torch.logsumexp(teacher / temperature, dim=1))
    weights = torch.full((tokens,), 1.0 / tokens, device="cuda")

    def logits_of(rows, h):  # h: the projections' output, or its 8-bit rows
        return (rows + down.forward(h, w_q)) @ w_head.t()

    def score(gate, up):
        return distill_forward(logits_of(x, block.forward(x, gate, up)), **lists)[0]

    result = {"quantized": float(score(w_gate, w_up).mean())}

    # 4. recovery of the projections in front of it (master weights in fp32)
    masters = [w_gate.float(), w_up.float()]
    kept = quantize_rows(x, group=128)
    for _ in range(steps):
        gate, up = (m.bfloat16() for m in masters)
        h = quantize_rows(block.forward(x, gate, up))
        logits = logits_of(x, h)
        _, d_logits = distill_step(logits, weights=weights, out=logits, **lists)  # over the logits
        d_h, _ = down.backward(d_logits @ w_head, h, w_q, want_dw=False)
        _, d_gate, d_up = block.backward(kept, gate, up, d_h, want_dx=False)
        for m, g in zip(masters, (d_gate, d_up)):
            m.sub_(g.float() * (lr * m.norm() / g.float().norm().clamp_min(1e-20) / 10))
    gate, up = (m.bfloat16() for m in masters)
    recovered = score(gate, up)
    result["recovered"] = float(recovered.mean())

    # 5. the same tokens one by one
    few = min(8, tokens)
    one = torch.cat([distill_forward(logits_of(x[t:t + 1], block.forward(x[t:t + 1], gate, up)),
                                     lists["top_logits"][t:t + 1], lists["top_index"][t:t + 1], temperature,
                                     lists["teacher_lse"][t:t + 1])[0] for t in range(few)])
    result["token_by_token"] = float(one.mean())
    result["same_tokens"] = float(recovered[:few].mean())
    block.sync()
    down.sync()
    hessian.sync()
    for handle in (block, down, hessian, gptq):
        handle.close()
    return result


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, value in (("d", 512), ("f", 1408), ("vocab", 4000), ("tokens", 2048), ("steps", 30)):
        ap.add_argument("--" + name, type=int, default=value)
    for key, value in run(**vars(ap.parse_args())).items():
        print(f"{key:16s} {value:.5f}")
