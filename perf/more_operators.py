"""Workloads of 8-bit rows, the 8-bit integer linear layer and backward passes from 8-bit checkpoints.

Each case is one pass through one operator as a program would call it:

* ``checkpoint``:  activations are kept as 8-bit rows and restored (``x -> codes,
  scales -> x^``): what a recovery step does with what its backward needs;
* ``linear``:      ``y[t, c] = sx[t] sw[c] sum_k qx[t, k] qw[c, k]`` with 16-bit
  activations that are quantized per token on the way and 8-bit weights with a
  scale per output channel: a quantized layer as it is served or evaluated;
* ``linear_grad``: that layer's gradients, straight through both roundings, from
  the 8-bit rows that its forward read;
* ``ff_grad``:     the gradients of the gated feed-forward projections with an
  8-bit checkpoint in the place of their input.

``own`` chooses between the plain form (elementary torch operations in 32
bits, rounded once at the end) and the framework's entry points.  ``exact``
states the same results in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ITEM = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # a decode batch's hidden states, a scale per token: latency
        rows("rows_few", 16, 4096, "f16", 0),
        # an odd ragged batch in fp32, a scale per 64 columns
        rows("rows_odd", 777, 2564, "f32", 64),
        # the feed-forward activations of a long training batch
        rows("rows_batch", 16384, 11008, "bf16", 128),
        # one token of a decode step: latency
        linear("linear_one_token", "linear", 1, 4096, 11008, "bf16"),
        # a decode batch of requests through the down projection, weights from HBM
        linear("linear_requests", "linear", 37, 11008, 4096, "f16"),
        # one ragged evaluation batch
        linear("linear_ragged", "linear", 777, 2560, 6912, "bf16"),
        # a full evaluation batch or prompt
        linear("linear_batch", "linear", 8192, 4096, 11008, "bf16"),
        # gradients of a narrow odd-sized layer
        linear("linear_grad_odd", "linear_grad", 203, 528, 1400, "f16"),
        # gradients of a down projection for a training batch
        linear("linear_grad_batch", "linear_grad", 4096, 11008, 4096, "bf16"),
        # gradients of a narrow odd-sized block from its checkpoint
        ff("ff_grad_odd", 203, 520, 1400, "f16", "gelu_tanh", 0),
        # gradients of a full block from its checkpoint for a training batch
        ff("ff_grad_batch", 4096, 4096, 11008, "bf16", "silu", 128),
    ]


def rows(name, n, d, dtype, group):
    return {"name": name, "op": "checkpoint", "tokens": n, "d": d, "dtype": dtype, "group": group}


def linear(name, op, n, d, f, dtype):
    return {"name": name, "op": op, "tokens": n, "d": d, "f": f, "dtype": dtype}


def ff(name, n, d, f, dtype, act, group):
    return {"name": name, "op": "ff_grad", "tokens": n, "d": d, "f": f, "dtype": dtype, "act": act, "group": group}


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["checkpoint", "linear", "linear", "linear_grad", "ff_grad"])
    if op == "checkpoint":
        n, d = log_int(4, 32768), log_int(64, 16384)
        dtype = rng.choice(["bf16", "f16", "f32"])
        n = max(1, min(n, (1 << 27) // d))
        case = rows("", n, d, dtype, rng.choice([0, 0, 32, 64, 128, 256]))
    elif op == "ff_grad":
        case = ff("", log_int(16, 4096), 8 * log_int(16, 512), 8 * log_int(32, 1376), rng.choice(["bf16", "f16"]),
                  rng.choice(["silu", "gelu_tanh"]), rng.choice([0, 64, 128]))
    else:
        d, f = 16 * log_int(8, 688), 8 * log_int(16, 1376)
        n = log_int(1, 8192) if op == "linear" else log_int(16, 4096)
        case = linear("", op, n, d, f, rng.choice(["bf16", "f16"]))
    del case["name"]
    return case


def to_rows8(x, group):
    """Codes and scales of fp32 values x [n, d]: a scale per row, or per `group` columns of a row.
    Quotients are taken in 64 bits, so that none is rounded onto a half."""
    n, d = x.shape
    if group == 0:
        top = x.abs().amax(dim=1, keepdim=True)
    else:
        top = torch.nn.functional.pad(x.abs(), (0, -d % group)).view(n, -1, group).amax(dim=2)
    s = (top.double() / 127.0).float()
    wide = s if group == 0 else s.repeat_interleave(group, dim=1)[:, :d]
    q = torch.where(wide > 0, torch.round(x.double() / wide.double()).float(), torch.zeros_like(x)).clamp(-127, 127)
    return q, s[:, 0] if group == 0 else s


def wide_scale(s, group, d):
    """The scale of every column, [n, d] or [n, 1]."""
    return s[:, None] if group == 0 else s.repeat_interleave(group, dim=1)[:, :d]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    n, d = case["tokens"], case["d"]
    s = {"case": case}
    x = torch.randn((n, d), generator=gen, device="cuda")
    x[:, torch.rand(d, generator=gen, device="cuda") < 0.01] *= 8.0  # outlier channels
    x *= 0.5 + torch.rand((n, 1), generator=gen, device="cuda")  # tokens of different size
    if n > 8:
        x[torch.randint(n, (1 + n // 64,), generator=gen, device="cuda")] = 0.0  # padding
    x = x.to(dt)
    if case["op"] == "checkpoint":
        s["x"] = x
        return s
    f = case["f"]
    if case["op"] == "ff_grad":
        q, s["scale"] = to_rows8(x.float(), case["group"])
        s["codes"] = q.to(torch.int8)
        for k in ("w_gate", "w_up"):
            s[k] = (torch.randn((f, d), generator=gen, device="cuda") / math.sqrt(d)).to(dt)
        s["dh"] = (0.1 * torch.randn((n, f), generator=gen, device="cuda")).to(dt)
    else:
        w = torch.randn((f, d), generator=gen, device="cuda") / math.sqrt(d)
        q, s["w_scale"] = to_rows8(w, 0)
        s["w_codes"] = q.to(torch.int8)
        if case["op"] == "linear":
            s["x"] = x
        else:
            q, s["scale"] = to_rows8(x.float(), 0)
            s["codes"] = q.to(torch.int8)
            s["dy"] = (0.1 * torch.randn((n, f), generator=gen, device="cuda")).to(dt)
    if own:
        from gptq_qqq_calibration_gb300 import GatedFF, Int8Linear, Rows8
        if case["op"] == "ff_grad":
            s["handle"] = GatedFF(d, f, train_tokens=n, dtype=dt, activation=case["act"], rows8=True)
            s["rows"] = Rows8(s["codes"], s["scale"], case["group"])
        else:
            s["handle"] = Int8Linear(d, f, tokens=n, train_tokens=n if case["op"] == "linear_grad" else 0, dtype=dt)
            s["weight"] = Rows8(s["w_codes"], s["w_scale"], 0)
            if case["op"] == "linear_grad":
                s["rows"] = Rows8(s["codes"], s["scale"], 0)
    return s


def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    case = s["case"]
    if case["op"] == "checkpoint":
        from gptq_qqq_calibration_gb300 import quantize_rows, restore_rows
        kept = quantize_rows(s["x"], group=case["group"])
        return {"scale": kept.scale, "x": restore_rows(kept, s["x"].dtype)}
    if case["op"] == "linear":
        return {"y": s["handle"].forward(s["x"], s["weight"])}
    if case["op"] == "linear_grad":
        dx, dw = s["handle"].backward(s["dy"], s["rows"], s["weight"])
        return {"dx": dx, "dw": dw}
    dx, dwg, dwu = s["handle"].backward(s["rows"], s["w_gate"], s["w_up"], s["dh"])
    return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}


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
    if case["op"] == "checkpoint":
        q, scale = to_rows8(s["x"].float(), case["group"])
        codes = q.to(torch.int8)
        return {"scale": scale, "x": (codes.float() * wide_scale(scale, case["group"], case["d"])).to(dt)}
    if case["op"] == "linear":
        q, scale = to_rows8(s["x"].float(), 0)
        return {"y": ((q @ s["w_codes"].float().t()) * (scale[:, None] * s["w_scale"][None, :])).to(dt)}
    if case["op"] == "linear_grad":
        x = s["codes"].float() * s["scale"][:, None]
        w = s["w_codes"].float() * s["w_scale"][:, None]
        dy = s["dy"].float()
        return {"dx": (dy @ w).to(dt), "dw": (dy.t() @ x).to(dt)}
    x = s["codes"].float() * wide_scale(s["scale"], case["group"], case["d"])
    wg, wu, dh = s["w_gate"].float(), s["w_up"].float(), s["dh"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, da = activation(g, case["act"])
    dg, du = dh * u * da, dh * a
    return {"dx": (dg @ wg + du @ wu).to(dt), "dw_gate": (dg.t() @ x).to(dt), "dw_up": (du.t() @ x).to(dt)}


def work(case):
    size, n, d = ITEM[case["dtype"]], case["tokens"], case["d"]
    groups = 1 if case.get("group", 0) == 0 else -(-d // case["group"])
    kept = n * d + 4 * n * groups
    if case["op"] == "checkpoint":  # x in and the rows out; the rows in and x^ out
        return {"bytes": 2 * (size * n * d + kept), "flops": 4 * n * d}
    f = case["f"]
    if case["op"] == "linear":
        return {"bytes": size * n * d + f * d + 4 * f + size * n * f, "flops": 2 * n * d * f}
    if case["op"] == "linear_grad":  # rows, weight and dy in; dx and dw out
        return {"bytes": kept + f * d + 4 * f + size * (n * f + n * d + f * d), "flops": 4 * n * d * f}
    # rows, both weights and dh in; dx and both weight gradients out
    return {"bytes": kept + size * (4 * f * d + n * f + n * d), "flops": 12 * n * d * f}


def exact_rows8(x, group):
    """Codes and per-column scales in 64 bits; a scale is a float32 number."""
    n, d = x.shape
    width = d if group == 0 else group
    parts = [x[:, a:a + width] for a in range(0, d, width)]
    scales = torch.stack([p.abs().max(dim=1).values.div(127).float().double() for p in parts], dim=1)
    at = torch.arange(d, device=x.device) // width
    full = scales[:, at]
    codes = torch.where(full == 0, 0.0, (x / full).round()).clamp(-127.0, 127.0)
    return codes, full, scales


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        codes, full, scales = exact_rows8(s["x"].double(), case["group"])
        return {"scale": scales[:, 0] if case["group"] == 0 else scales, "x": codes * full}
    n, d, f = case["tokens"], case["d"], case["f"]
    if (12 if case["op"] == "ff_grad" else 4) * n * d * f > 5e12:
        return None
    if case["op"] == "linear":
        codes, full, _ = exact_rows8(s["x"].double(), 0)
        y = torch.matmul(codes, s["w_codes"].double().T)
        return {"y": y * full[:, :1] * s["w_scale"].double()}
    group = case.get("group", 0)
    at = torch.arange(d, device="cuda") // (d if group == 0 else group)
    x = s["codes"].double() * s["scale"].double().reshape(n, -1)[:, at]
    if case["op"] == "linear_grad":
        dy = s["dy"].double()
        w = s["w_scale"].double()[:, None] * s["w_codes"].double()
        return {"dx": torch.matmul(dy, w), "dw": torch.matmul(dy.T, x)}
    wg, wu, dh = (s[k].double() for k in ("w_gate", "w_up", "dh"))
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
    dup, dgate = dh * value, dh * up * slope
    return {"dx": torch.addmm(torch.matmul(dup, wu), dgate, wg), "dw_gate": torch.matmul(dgate.T, x),
            "dw_up": torch.matmul(dup.T, x)}
