"""Workloads of the gated feed-forward projections and of the distillation loss.

Each case is one pass through one operator as a program would call it:

* ``ff_forward``:   h = act(x Wg^T) * (x Wu^T), the input of a block's down
  projection (the activations whose Hessian a calibration collects);
* ``ff_backward``:  the gradients of x, Wg and Wu from the gradient of h;
* ``distill_loss``: per-row divergence of a student's full logits from a
  teacher's top logits (evaluation of a quantized model against its original);
* ``distill_step``: that loss and the gradient of the student's logits in one
  call (a recovery step whose row weights already hold the mean's 1/n);
* ``distill_grad``: the loss, then the gradient under a given gradient of the
  row losses (what an autograd graph around the loss runs).

``own`` chooses between the plain form (elementary torch operations in 32
bits, rounded once at the end) and the framework's entry points.  ``exact``
states the same results in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ITEM = {"bf16": 2, "f16": 2, "f32": 4}

# Rows without weight (prompt tokens, padding) and rows whose teacher entries
# are all empty, as shares of the rows of a distillation batch.
MASKED, EMPTY = 0.125, 0.03


def listed():
    return [
        # one token of a decode step through a small block: latency
        ff("ff_fwd_one_token", "ff_forward", 1, 2560, 6912, "bf16", "silu"),
        # a decode batch of requests, weights from HBM
        ff("ff_fwd_requests", "ff_forward", 37, 4096, 11008, "f16", "silu"),
        # one ragged calibration batch
        ff("ff_fwd_ragged", "ff_forward", 777, 2560, 6912, "bf16", "gelu_tanh"),
        # a full calibration batch or prompt
        ff("ff_fwd_batch", "ff_forward", 8192, 4096, 11008, "bf16", "silu"),
        # a narrow odd-sized block under training
        ff("ff_bwd_odd", "ff_backward", 203, 520, 1400, "f16", "gelu_tanh"),
        # a training batch through a full block
        ff("ff_bwd_batch", "ff_backward", 4096, 4096, 11008, "bf16", "silu"),
        # scoring the next-token logits of a few sequences
        distill("distill_loss_few", "distill_loss", 4, 32000, 32, "f32", 1.0, False),
        # scoring a batch of a quantized model's logits, full-mass teacher
        distill("distill_loss_batch", "distill_loss", 2048, 131072, 64, "bf16", 1.0, True),
        # one recovery step on a small batch with an odd vocabulary
        distill("distill_step_odd", "distill_step", 301, 50257, 100, "f32", 2.0, True),
        # one recovery step on a full batch
        distill("distill_step_batch", "distill_step", 8192, 128000, 64, "bf16", 1.0, False),
        # the loss under autograd, small
        distill("distill_grad_small", "distill_grad", 64, 32001, 16, "f16", 1.5, False),
        # the loss under autograd, a full batch
        distill("distill_grad_batch", "distill_grad", 4096, 65536, 128, "bf16", 2.0, True),
    ]


def ff(name, op, tokens, d, f, dtype, act):
    return {"name": name, "op": op, "tokens": tokens, "d": d, "f": f, "dtype": dtype, "act": act}


def distill(name, op, rows, vocab, top, dtype, temperature, full_mass):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "top": top, "dtype": dtype,
            "temperature": temperature, "full_mass": full_mass}


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["ff_forward", "ff_forward", "ff_backward", "distill_loss", "distill_step", "distill_grad"])
    if op.startswith("ff"):
        d, f = 8 * log_int(16, 512), 8 * log_int(32, 1376)
        tokens = log_int(1 if op == "ff_forward" else 16, 8192 if op == "ff_forward" else 4096)
        case = ff("", op, tokens, d, f, rng.choice(["bf16", "f16"]), rng.choice(["silu", "gelu_tanh"]))
    else:
        rows, vocab = log_int(4, 8192), log_int(4000, 160000)
        rows = min(rows, 8192 * 128000 // vocab)
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if dtype == "f32":
            rows = max(1, rows // 2)
        case = distill("", op, rows, vocab, log_int(4, 256), dtype, rng.choice([0.75, 1.0, 1.5, 2.0, 3.0]),
                       rng.choice([False, True]))
    del case["name"]
    return case


def live_rows(case):
    """Rows with weight and with teacher entries; the others come first."""
    return case["rows"] - int(MASKED * case["rows"]) - int(EMPTY * case["rows"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"].startswith("ff"):
        n, d, f = case["tokens"], case["d"], case["f"]
        x = torch.randn((n, d), generator=gen, device="cuda")
        x[:, torch.rand(d, generator=gen, device="cuda") < 0.01] *= 8.0  # outlier channels
        s["x"] = x.to(dt)
        for k in ("w_gate", "w_up"):
            s[k] = (torch.randn((f, d), generator=gen, device="cuda") / math.sqrt(d)).to(dt)
        if case["op"] == "ff_backward":
            s["dh"] = (0.1 * torch.randn((n, f), generator=gen, device="cuda")).to(dt)
        if own:
            from gptq_qqq_calibration_gb300 import GatedFF
            s["ff"] = GatedFF(d, f, train_tokens=n if case["op"] == "ff_backward" else 0, dtype=dt,
                              activation=case["act"])
        return s
    rows, vocab, top = case["rows"], case["vocab"], min(case["top"], case["vocab"])
    logits = torch.empty((rows, vocab), dtype=dt, device="cuda")
    t_vals = torch.empty((rows, top), dtype=torch.float32, device="cuda")
    t_idx = torch.empty((rows, top), dtype=torch.int32, device="cuda")
    t_lse = torch.empty(rows, dtype=torch.float32, device="cuda")
    inv_t = 1.0 / case["temperature"]
    step = max(1, (1 << 28) // vocab)
    for a in range(0, rows, step):  # bounded temporaries
        b = min(rows, a + step)
        teacher = 2.5 * torch.randn((b - a, vocab), generator=gen, device="cuda")
        # a few likely tokens a row hold most of the mass
        at = torch.randint(vocab, (b - a, 32), generator=gen, device="cuda")
        teacher.scatter_add_(1, at, 8.0 + 6.0 * torch.rand((b - a, 32), generator=gen, device="cuda"))
        logits[a:b] = (teacher + 1.2 * torch.randn((b - a, vocab), generator=gen, device="cuda")).to(dt)
        v, i = torch.topk(teacher, top, dim=1)
        t_vals[a:b], t_idx[a:b] = v, i.to(torch.int32)
        t_lse[a:b] = torch.logsumexp(teacher * inv_t, dim=1)
    # an eighth of the rows has a teacher list that ends early
    short = torch.rand(rows, generator=gen, device="cuda") < 0.125
    t_idx[:, top // 2:][short] = -1
    masked, empty = int(MASKED * rows), int(EMPTY * rows)
    t_idx[masked:masked + empty] = -1
    weights = torch.full((rows,), 1.0 / max(1, rows - masked), dtype=torch.float32, device="cuda")
    weights[:masked] = 0.0
    s.update(logits=logits, top_logits=t_vals, top_index=t_idx, weights=weights,
             teacher_lse=t_lse if case["full_mass"] else None)
    if case["op"] == "distill_grad":
        s["grad"] = 0.5 + torch.rand(rows, generator=gen, device="cuda")
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    case = s["case"]
    if case["op"] == "ff_forward":
        return {"h": s["ff"].forward(s["x"], s["w_gate"], s["w_up"])}
    if case["op"] == "ff_backward":
        dx, dwg, dwu = s["ff"].backward(s["x"], s["w_gate"], s["w_up"], s["dh"])
        return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}
    from gptq_qqq_calibration_gb300 import distill_backward, distill_forward, distill_step
    teacher = dict(top_logits=s["top_logits"], top_index=s["top_index"], temperature=case["temperature"],
                   teacher_lse=s["teacher_lse"], weights=s["weights"])
    if case["op"] == "distill_step":
        loss, dlogits = distill_step(s["logits"], **teacher)
        return {"loss": loss, "dlogits": dlogits}
    loss, stats = distill_forward(s["logits"], **teacher)
    if case["op"] == "distill_loss":
        return {"loss": loss}
    return {"loss": loss, "dlogits": distill_backward(s["logits"], stats, grad=s["grad"], **teacher)}


def activation(g, kind):
    """act(g) and its derivative."""
    if kind == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        return g * sig, sig * (1.0 + g * (1.0 - sig))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def run_plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"].startswith("ff"):
        x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
        g, u = x @ wg.t(), x @ wu.t()
        a, da = activation(g, case["act"])
        if case["op"] == "ff_forward":
            return {"h": (a * u).to(dt)}
        dh = s["dh"].float()
        dg, du = dh * u * da, dh * a
        return {"dx": (dg @ wg + du @ wu).to(dt), "dw_gate": (dg.t() @ x).to(dt), "dw_up": (du.t() @ x).to(dt)}

    tau = case["temperature"]
    w = s["weights"]
    idx = s["top_index"].long()
    held = idx >= 0
    at = idx.clamp(min=0)
    live = held.any(dim=1, keepdim=True)
    full = s["teacher_lse"] is not None
    # student
    x = s["logits"].float()
    m = x.max(dim=1, keepdim=True).values
    e = torch.exp((x - m) / tau)
    total = e.sum(dim=1, keepdim=True)
    # teacher, and log(p / q) from the differences of like terms
    t = s["top_logits"]
    gap = (t - torch.gather(x, 1, at)) / tau
    if full:
        log_p = t / tau - s["teacher_lse"][:, None]
        p = torch.where(held, torch.exp(log_p), torch.zeros_like(t))
        gap = gap + (m / tau - s["teacher_lse"][:, None]) + torch.log(total)
    else:
        tm = torch.where(held, t, torch.full_like(t, -math.inf)).max(dim=1, keepdim=True).values
        tm = torch.where(live, tm, torch.zeros_like(tm))
        p = torch.where(held, torch.exp((t - tm) / tau), torch.zeros_like(t))
        t_total = torch.where(live, p.sum(dim=1, keepdim=True), torch.ones_like(tm))
        p = p / t_total
        gap = gap + (m - tm) / tau + torch.log(total) - torch.log(t_total)
    loss = torch.where(held & (p > 0), p * gap, torch.zeros_like(p)).sum(dim=1)
    rest = None
    if full:
        top = torch.zeros_like(e).scatter_add_(1, at, held.float()) > 0
        tail = torch.where(top, torch.zeros_like(e), e).sum(dim=1, keepdim=True) / total
        p_tail = (1.0 - p.sum(dim=1, keepdim=True)).clamp(min=0.0)
        some = p_tail > 0
        loss = loss + torch.where(some, p_tail * torch.log(p_tail / tail), torch.zeros_like(tail))[:, 0]
        rest = torch.where(some, 1.0 - p_tail / tail, torch.ones_like(tail))
    use = live[:, 0] & (w != 0)
    loss = torch.where(use, loss * w * (tau * tau), torch.zeros_like(loss))
    if case["op"] == "distill_loss":
        return {"loss": loss}
    q = e / total
    if rest is not None:
        q = torch.where(top, q, q * rest)
    q.scatter_add_(1, at, -p)
    scale = w * tau
    if case["op"] == "distill_grad":
        scale = scale * s["grad"]
    q = torch.where(use[:, None], q * scale[:, None], torch.zeros_like(q[:1, :1]))
    return {"loss": loss, "dlogits": q.to(dt)}


def work(case):
    size = ITEM[case["dtype"]]
    if case["op"].startswith("ff"):
        n, d, f = case["tokens"], case["d"], case["f"]
        if case["op"] == "ff_forward":
            return {"bytes": size * (n * d + 2 * f * d + n * f), "flops": 4 * n * d * f}
        # x, both weights and dh in; dx and both weight gradients out.  The
        # projections, the gradient of x and those of the weights: 4 n d f each.
        return {"bytes": size * (2 * n * d + 4 * f * d + n * f), "flops": 12 * n * d * f}
    rows, live, vocab = case["rows"], live_rows(case), case["vocab"]
    lists = live * (8 * min(case["top"], vocab) + 4) + 8 * rows
    if case["op"] == "distill_loss":
        return {"bytes": size * live * vocab + lists, "flops": 4 * live * vocab}
    return {"bytes": size * (live + rows) * vocab + lists, "flops": 7 * live * vocab}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("ff"):
        n, d, f = case["tokens"], case["d"], case["f"]
        if 12 * n * d * f > 5e12:
            return None
        return exact_ff(s, case)
    return exact_distill(s, case)


def exact_ff(s, case):
    x, wg, wu = (s[k].double() for k in ("x", "w_gate", "w_up"))
    gate, up = torch.matmul(x, wg.T), torch.matmul(x, wu.T)
    if case["act"] == "silu":
        value = gate * torch.sigmoid(gate)
        slope = torch.sigmoid(gate) + value * torch.sigmoid(-gate)
    else:
        # 0.5 (1 + tanh y) = sigmoid(2 y)
        y2 = 2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)
        half = torch.sigmoid(y2)
        value = gate * half
        slope = half + value * torch.sigmoid(-y2) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * gate ** 2)
    if case["op"] == "ff_forward":
        return {"h": value * up}
    dh = s["dh"].double()
    dup = dh * value
    dgate = dh * up * slope
    return {"dx": torch.addmm(torch.matmul(dup, wu), dgate, wg), "dw_gate": torch.matmul(dgate.T, x),
            "dw_up": torch.matmul(dup.T, x)}


def exact_distill(s, case):
    rows, vocab, tau = case["rows"], case["vocab"], case["temperature"]
    losses = torch.zeros(rows, dtype=torch.float64, device="cuda")
    want_grad = case["op"] != "distill_loss"
    grads = torch.zeros((rows, vocab), dtype=torch.float64, device="cuda") if want_grad else None
    step = max(1, (1 << 27) // vocab)
    for a in range(0, rows, step):
        b = min(rows, a + step)
        log_q = torch.log_softmax(s["logits"][a:b].double() / tau, dim=1)
        idx = s["top_index"][a:b].long()
        t = s["top_logits"][a:b].double() / tau
        t = t.masked_fill(idx < 0, -math.inf)
        # the teacher's list as one more column: a place that collects empties
        place = torch.where(idx < 0, vocab, idx)
        if case["full_mass"]:
            logp = t - s["teacher_lse"][a:b, None].double()
        else:
            logp = t - torch.logsumexp(t, dim=1, keepdim=True)
        logp = torch.where(idx < 0, -math.inf, logp)
        p = logp.exp()
        wide = torch.cat([log_q, torch.zeros((b - a, 1), dtype=torch.float64, device="cuda")], dim=1)
        terms = p * (logp - wide.gather(1, place))
        row = torch.where(p > 0, terms, 0.0).sum(1)
        target = torch.zeros((b - a, vocab + 1), dtype=torch.float64, device="cuda").scatter_add(1, place, p)[:, :vocab]
        factor = None
        if case["full_mass"]:
            hit = torch.zeros((b - a, vocab + 1), dtype=torch.bool, device="cuda").scatter(1, place, True)[:, :vocab]
            p_rest = 1.0 - p.sum(1)
            logq_rest = torch.logsumexp(log_q.masked_fill(hit, -math.inf), dim=1)
            some = p_rest > 0
            row = row + torch.where(some, p_rest * (torch.log(p_rest) - logq_rest), 0.0)
            factor = torch.where(some, 1.0 - p_rest / logq_rest.exp(), 1.0)
        w = s["weights"][a:b].double()
        use = (w != 0) & (idx >= 0).any(1)
        losses[a:b] = torch.where(use, tau * tau * w * row, 0.0)
        if want_grad:
            q = log_q.exp()
            if factor is not None:
                q = torch.where(hit, q, q * factor[:, None])
            scale = tau * w * (s["grad"][a:b].double() if case["op"] == "distill_grad" else 1.0)
            grads[a:b] = torch.where(use[:, None], (q - target) * scale[:, None], 0.0)
    return {"loss": losses, "dlogits": grads} if want_grad else {"loss": losses}
