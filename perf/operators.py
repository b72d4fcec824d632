"""The output head's operators: what is measured of them, and their plain forms.

Two families that stand beside the ternary layers of this library:

- ``fp8_quant``, ``fp8_linear``, ``fp8_train``: a linear layer in 8-bit floating point
  with one power-of-two scale for each block of 128 along the reduction (1 x 128 blocks
  of activations and gradients, 128 x 128 blocks of weights), for the projections that a
  ternary model keeps in higher precision;
- ``ce_fwd``, ``ce_train``: softmax cross entropy over a large vocabulary straight from
  the hidden states and the head's weights, and its gradients, without the logits.

Layouts shared by both forms: codes of a [rows, cols] tensor are float8 [rows, cols];
their scales are uint8 exponents [ceil(cols / 512), rows, 4] (block b of row r at
[b // 4, r, b % 4], scale 2^(byte - 127), bytes of blocks past the end 0). The transposed
copy of a [t, k] tensor is [k, t rounded up to 16], zero behind t, with blocks along t.
"""
import torch

own = False

E4M3, E5M2 = "float8_e4m3fn", "float8_e5m2"
TOP = {E4M3: 8, E5M2: 15}          # the largest finite value is 1.75 * 2^TOP
LINEAR_MOST = 16384 * 2048 * 11008   # t * k * n of the largest linear case
HEAD_MOST = 8192 * 65536 * 2048      # t * v * k of the largest head case


def listed():
    return [
        # one token through a down projection: latency and the stream of its weights
        {"name": "fp8_linear_t1_11008x2048", "op": "fp8_linear", "t": 1, "k": 11008, "n": 2048},
        # a decode batch through a gate projection
        {"name": "fp8_linear_t32_2048x11008", "op": "fp8_linear", "t": 32, "k": 2048, "n": 11008},
        # a prompt of odd length
        {"name": "fp8_linear_t777_1536x8960", "op": "fp8_linear", "t": 777, "k": 1536, "n": 8960},
        # prefill
        {"name": "fp8_linear_t8192_2048x11008", "op": "fp8_linear", "t": 8192, "k": 2048, "n": 11008},
        # a training step of a small down projection, ragged tokens, gradients in e5m2
        {"name": "fp8_train_t4095_4864x896", "op": "fp8_train", "t": 4095, "k": 4864, "n": 896, "dy": E5M2},
        # a training step of a large gate projection: weights and activations quantised, three products
        {"name": "fp8_train_t16384_2048x11008", "op": "fp8_train", "t": 16384, "k": 2048, "n": 11008, "dy": E4M3},
        # the activations of that layer's successor, for its forward product and its weight gradient
        {"name": "fp8_quant_t16384_11008", "op": "fp8_quant", "what": "activations", "t": 16384, "k": 11008, "fmt": E4M3},
        # the weights after an optimizer step, for the forward product and the input gradient
        {"name": "fp8_quant_w11008x2048", "op": "fp8_quant", "what": "weights", "t": 11008, "k": 2048, "fmt": E4M3},
        # the log-probability of one token
        {"name": "ce_fwd_t1_v32768_2048", "op": "ce_fwd", "t": 1, "k": 2048, "v": 32768},
        # scoring a text of ordinary length over an odd vocabulary
        {"name": "ce_fwd_t1000_v50001_896", "op": "ce_fwd", "t": 1000, "k": 896, "v": 50001},
        # a training step over a ragged batch and an odd vocabulary
        {"name": "ce_train_t2047_v32003_1536", "op": "ce_train", "t": 2047, "k": 1536, "v": 32003},
        # a training step at full size
        {"name": "ce_train_t8192_v65536_2048", "op": "ce_train", "t": 8192, "k": 2048, "v": 65536},
    ]


def _spread(rng, low, high, step=1):
    """A multiple of ``step`` in [low, high], spread over its logarithm."""
    v = low * (high / low) ** rng.random()
    return max(low, min(high, int(v) // step * step))


def draw(rng):
    op = rng.choice(["fp8_linear", "fp8_linear", "fp8_train", "fp8_quant", "ce_fwd", "ce_train"])
    t = _spread(rng, 1, 16384)
    k = _spread(rng, 64, 11008, 64)
    if op.startswith("ce"):
        t = min(t, 8192)
        v = _spread(rng, 500, 131072)
        while t * v * k > HEAD_MOST or v * k > 65536 * 2048:
            t, v = max(1, t // 2), max(500, v * 3 // 4)
        return {"op": op, "t": t, "k": k, "v": v}
    if op == "fp8_quant":
        what = rng.choice(["activations", "weights"])
        t = _spread(rng, 16, 11008, 16) if what == "weights" else t
        return {"op": op, "what": what, "t": t, "k": k, "fmt": rng.choice([E4M3, E5M2])}
    n = _spread(rng, 16, 11008, 16)
    while t * k * n > LINEAR_MOST:
        t = max(1, t // 2)
    case = {"op": op, "t": t, "k": k, "n": n}
    if op == "fp8_train":
        case["dy"] = rng.choice([E4M3, E5M2])
    return case


# ------------------------------------------------------------------ inputs

def _rand(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * std


def _activations(gen, t, k):
    """bf16 hidden states: N(0, 1) with 1% of the entries 20 times as large."""
    x = _rand(gen, t, k)
    big = torch.rand(t, k, generator=gen, device="cuda") < 0.01
    return torch.where(big, x * 20.0, x).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, t, k = case["op"], case["t"], case["k"]
    if op == "fp8_quant":
        src = _activations(gen, t, k) if case["what"] == "activations" else _rand(gen, t, k, std=0.02)
        return {**case, "src": src}
    if op == "fp8_linear":
        w = _quantised(_rand(gen, case["n"], k, std=0.02), 128, E4M3)   # laid out once, as a server does
        return {**case, "x": _activations(gen, t, k), "w": w}
    if op == "fp8_train":
        return {**case, "x": _activations(gen, t, k), "dy_in": _rand(gen, t, case["n"], std=1e-2).to(torch.bfloat16),
                "w": _rand(gen, case["n"], k, std=0.02)}
    v = case["v"]
    w = _rand(gen, v, k, std=0.02).to(torch.bfloat16)
    targets = torch.randint(0, v, (t,), generator=gen, device="cuda")
    # hidden states that know their target to a varying degree, so that losses run from near 0 to log v
    push = torch.rand(t, 1, generator=gen, device="cuda") * 12.0
    row = w[targets].float()
    x = (_rand(gen, t, k) + push * row / (row * row).sum(1, keepdim=True)).to(torch.bfloat16)
    if t > 8:   # padding and prompt positions carry no loss
        targets = torch.where(torch.rand(t, generator=gen, device="cuda") < 0.06, -100, targets)
    weight = torch.full((t,), 1.0 / t, device="cuda")   # the gradient of a mean over the tokens
    return {**case, "x": x, "w": w, "targets": targets, "weight": weight}


# ------------------------------------------------------------------ plain forms

def _quantised(x, rows, fmt):
    """Codes and scale exponents of x in blocks of ``rows`` x 128 (``rows`` 1 or 128)."""
    r, c = x.shape
    pad_r, pad_c = -r % rows, -c % 512
    p = torch.nn.functional.pad(x.float(), (0, pad_c, 0, pad_r))
    blocks = p.reshape((r + pad_r) // rows, rows, (c + pad_c) // 128, 128)
    m, e = torch.frexp(blocks.abs().amax(dim=(1, 3)))        # amax = m * 2^e, 0.5 <= m < 1
    byte = (e - 1 - TOP[fmt] + (m > 0.875).int() + 127).clamp(0, 254)
    byte = torch.where(m == 0, 0, byte)
    scaled = torch.ldexp(blocks, (127 - byte)[:, None, :, None])
    codes = scaled.reshape(r + pad_r, c + pad_c)[:r, :c].to(getattr(torch, fmt))
    per_row = byte.to(torch.uint8).repeat_interleave(rows, 0)[:r]
    return codes.contiguous(), per_row.reshape(r, -1, 4).permute(1, 0, 2).contiguous()


def _both(x, rows, fmt):
    """Codes and scales along the rows, and of the transposed copy padded to 16."""
    q, s = _quantised(x, rows, fmt)
    turned = torch.nn.functional.pad(x.t(), (0, -x.shape[0] % 16)).contiguous()
    qt, st = _quantised(turned, rows, fmt)
    return q, s, qt, st


def _values(q, s):
    """What codes and scales stand for, in 32 bits."""
    r, c = q.shape
    exponent = (s.permute(1, 0, 2).reshape(r, -1).int() - 127).repeat_interleave(128, 1)[:, :c]
    return torch.ldexp(q.float(), exponent)


def _plain_ce(x, w, targets):
    logits = x.float() @ w.float().t()
    counts = (targets >= 0) & (targets < w.shape[0])
    at = torch.where(counts, targets, 0)
    top = logits.amax(1, keepdim=True)
    lse = (top + (logits - top).exp().sum(1, keepdim=True).log())[:, 0]
    loss = torch.where(counts, lse - logits.gather(1, at[:, None])[:, 0], 0.0)
    return logits, counts, at, lse, loss


def run(state):
    op = state["op"]
    if own:
        return _run_own(op, state)
    if op == "fp8_quant":
        return _both(state["src"], 1 if state["what"] == "activations" else 128, state["fmt"])
    if op == "fp8_linear":
        return (_values(*_quantised(state["x"], 1, E4M3)) @ _values(*state["w"]).t()).to(torch.bfloat16)
    if op == "fp8_train":
        xq, xs, xt, xts = _both(state["x"], 1, E4M3)
        dq, ds, dt, dts = _both(state["dy_in"], 1, state["dy"])
        wq, ws = _quantised(state["w"], 128, E4M3)
        w = _values(wq, ws)
        y = _values(xq, xs) @ w.t()
        grad_x = _values(dq, ds) @ w
        grad_w = _values(dt, dts) @ _values(xt, xts).t()
        return y.to(torch.bfloat16), grad_x.to(torch.bfloat16), grad_w.to(torch.bfloat16)
    x, w = state["x"], state["w"]
    logits, counts, at, lse, loss = _plain_ce(x, w, state["targets"])
    if op == "ce_fwd":
        return loss, lse
    g = torch.where(counts, state["weight"], 0.0)[:, None]
    d = (logits - lse[:, None]).exp_()
    d.scatter_add_(1, at[:, None], torch.full_like(g, -1.0))
    d *= g
    return loss, lse, (d @ w.float()).to(torch.bfloat16), (d.t() @ x.float()).to(torch.bfloat16)


def _run_own(op, state):
    import sparsity_step_b200 as B

    if op == "fp8_quant":
        fmt = getattr(torch, state["fmt"])
        q = (B.bitlinear_fp8_quant if state["what"] == "activations" else B.bitlinear_fp8_quant_weight)(
            state["src"], want_t=True, fmt=fmt)
        return q["q"], q["scales"], q["qt"], q["scales_t"]
    if op == "fp8_linear":
        return B.bitlinear_fp8_fwd(state["x"], *state["w"])
    if op == "fp8_train":
        w = B.bitlinear_fp8_quant_weight(state["w"], want_t=True)
        x = B.bitlinear_fp8_quant(state["x"], want_t=True)
        y = B.bitlinear_fp8_fwd(x["q"], w["q"], w["scales"], x_scales=x["scales"])
        dy = B.bitlinear_fp8_quant(state["dy_in"], want_t=True, fmt=getattr(torch, state["dy"]))
        grad_x, grad_w = B.bitlinear_fp8_bwd(dy, x, w)
        return y, grad_x, grad_w
    loss, lse = B.bitlinear_linear_ce_fwd(state["x"], state["w"], state["targets"])
    if op == "ce_fwd":
        return loss, lse
    grad_x, grad_w = B.bitlinear_linear_ce_bwd(state["x"], state["w"], state["targets"], lse, state["weight"])
    return loss, lse, grad_x, grad_w


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, t, k = case["op"], case["t"], case["k"]
    if op == "fp8_quant":
        size = 2 if case["what"] == "activations" else 4
        return {"bytes": t * k * (size + 2) + 2 * t * k // 128, "flops": 4 * t * k}
    if op.startswith("fp8"):
        n = case["n"]
        if op == "fp8_linear":
            return {"bytes": 2 * t * k + n * k + n * k // 128 + 2 * t * n, "flops": 2 * t * k * n}
        return {"bytes": 2 * t * k + 2 * t * n + 4 * n * k + 2 * t * n + 2 * t * k + 2 * n * k, "flops": 6 * t * k * n}
    v = case["v"]
    if op == "ce_fwd":
        return {"bytes": 2 * t * k + 2 * v * k + 16 * t, "flops": 2 * t * v * k}
    return {"bytes": 4 * t * k + 4 * v * k + 20 * t, "flops": 6 * t * v * k}


# ------------------------------------------------------------------ 64 bits, from the definitions

def _round_to(v, fmt):
    """v (64 bits, within the format's range) at the format's nearest value, ties to even."""
    bits, low = (3, -6) if fmt == E4M3 else (2, -14)
    step = torch.exp2((torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -40))).clamp_min(low) - bits))
    return torch.round(v / step) * step


def _exact_quantised(x, rows, fmt):
    """(codes, scales, values) with each block's scale found by comparison: the smallest
    power of two that brings the block within the format."""
    x = x.double()
    r, c = x.shape
    limit = 1.75 * 2.0 ** TOP[fmt]
    nb = (c + 127) // 128
    amax = torch.stack([x[:, 128 * b:128 * (b + 1)].abs().amax(1) for b in range(nb)], 1)   # [r, nb]
    if rows > 1:
        per = torch.stack([amax[i:i + rows].amax(0) for i in range(0, r, rows)], 0)
        amax = per[torch.arange(r, device=x.device) // rows]
    e = torch.ceil(torch.log2((amax / limit).clamp_min(2.0 ** -200)))
    e = torch.where(torch.exp2(e) * limit < amax, e + 1, e)
    e = torch.where(torch.exp2(e - 1) * limit >= amax, e - 1, e).clamp(-127, 127)
    block = torch.arange(c, device=x.device) // 128
    scale = torch.exp2(e)[:, block]
    codes = _round_to(x / scale, fmt)
    scales = torch.zeros((c + 511) // 512, r, 4, dtype=torch.uint8, device=x.device)
    for b in range(nb):
        scales[b // 4, :, b % 4] = (e[:, b] + 127).to(torch.uint8)
    return codes, scales, codes * scale


def _turned(x):
    out = torch.zeros(x.shape[1], (x.shape[0] + 15) // 16 * 16, dtype=torch.float64, device=x.device)
    out[:, :x.shape[0]] = x.double().t()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "fp8_quant":
        rows = 1 if case["what"] == "activations" else 128
        q, sc, _ = _exact_quantised(s["src"], rows, case["fmt"])
        qt, sct, _ = _exact_quantised(_turned(s["src"]), rows, case["fmt"])
        return q, sc, qt, sct
    if op == "fp8_linear":
        wq, ws = s["w"]
        w = wq.double()
        for b in range((case["k"] + 127) // 128):
            w[:, 128 * b:128 * (b + 1)] *= torch.exp2(ws[b // 4, :, b % 4].double() - 127)[:, None]
        return _exact_quantised(s["x"], 1, E4M3)[2] @ w.t()
    if op == "fp8_train":
        w = _exact_quantised(s["w"], 128, E4M3)[2]
        y = _exact_quantised(s["x"], 1, E4M3)[2] @ w.t()
        grad_x = _exact_quantised(s["dy_in"], 1, case["dy"])[2] @ w
        grad_w = (_exact_quantised(_turned(s["dy_in"]), 1, case["dy"])[2]
                  @ _exact_quantised(_turned(s["x"]), 1, E4M3)[2].t())
        return y, grad_x, grad_w
    x, w, targets = s["x"].double(), s["w"].double(), s["targets"]
    p = x @ w.t()
    lse = torch.logsumexp(p, 1)
    rows = torch.arange(case["t"], device=p.device)
    live = (targets >= 0) & (targets < case["v"])
    at = targets.clamp(0, case["v"] - 1)
    loss = torch.where(live, lse - p[rows, at], torch.zeros_like(lse))
    if op == "ce_fwd":
        return loss, lse
    p = p.sub_(lse[:, None]).exp_()
    p[rows, at] -= 1.0
    p *= torch.where(live, s["weight"].double(), torch.zeros_like(lse))[:, None]
    return loss, lse, p @ w, p.t() @ x
