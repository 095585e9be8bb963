"""Operators of a transformer's feed-forward half layer: cases to measure.

Four operators are called here, in the order a layer meets them: layer norm
(forward, or forward and backward), the gated feed-forward projections
h = act(x Wg^T) * (x Wu^T) (forward, or forward and backward), the 8-bit integer
product with a scale per token and per channel, and that product fed by the
quantisation of 16-bit activations token by token.

`run` computes a case in elementary torch operations, or, where `own` is true,
through the kernels of this package.  `exact` computes the definition again in
binary64.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of a decode step through the norm: latency only
        {"name": "norm_1x8192_bf16", "op": "norm", "rows": 1, "cols": 8192, "dtype": "bf16",
         "wdtype": "bf16", "train": False},
        # a long prefill's activations: one read and one write of 268 MB
        {"name": "norm_16384x8192_bf16", "op": "norm", "rows": 16384, "cols": 8192,
         "dtype": "bf16", "wdtype": "bf16", "train": False},
        # a training step on ragged rows (odd length: rows start 2-byte aligned),
        # fp16 activations with fp32 master weights
        {"name": "norm_train_4097x3001_f16", "op": "norm", "rows": 4097, "cols": 3001,
         "dtype": "f16", "wdtype": "f32", "train": True},
        # a training step over a large batch of tokens
        {"name": "norm_train_16384x4096_bf16", "op": "norm", "rows": 16384, "cols": 4096,
         "dtype": "bf16", "wdtype": "bf16", "train": True},
        # one token of a decode step: both weights are read once
        {"name": "gated_1x7168x4096_bf16", "op": "gated", "rows": 1, "hidden": 7168,
         "cols": 4096, "dtype": "bf16", "act": "silu", "train": False},
        # a decode batch of 64 tokens on 8192-wide weights
        {"name": "gated_64x8192x8192_f16", "op": "gated", "rows": 64, "hidden": 8192,
         "cols": 8192, "dtype": "f16", "act": "gelu_tanh", "train": False},
        # a training step on ragged sizes
        {"name": "gated_train_1027x2003x1501_f16", "op": "gated", "rows": 1027, "hidden": 2003,
         "cols": 1501, "dtype": "f16", "act": "gelu", "train": True},
        # a training step of 4096 tokens: the largest case
        {"name": "gated_train_4096x7168x4096_bf16", "op": "gated", "rows": 4096, "hidden": 7168,
         "cols": 4096, "dtype": "bf16", "act": "silu", "train": True},
        # one decoded token, activations already in 8 bits
        {"name": "i8_1x8192x8192_bf16", "op": "i8", "rows": 1, "n": 8192, "k": 8192,
         "out": "bf16", "quantise": False},
        # a prefill's product, activations already in 8 bits
        {"name": "i8_8192x8192x8192_bf16", "op": "i8", "rows": 8192, "n": 8192, "k": 8192,
         "out": "bf16", "quantise": False},
        # ragged rows: a decode batch quantised on the way in
        {"name": "i8_quantise_77x3001x5003_f16", "op": "i8", "rows": 77, "n": 3001, "k": 5003,
         "out": "f16", "quantise": True},
        # a prefill chunk quantised on the way in
        {"name": "i8_quantise_4096x7168x4096_bf16", "op": "i8", "rows": 4096, "n": 7168,
         "k": 4096, "out": "bf16", "quantise": True},
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of lo..hi; half of them a multiple of a
    power of two as widths mostly are, the others any number, odd ones too."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        step = 1 << max(0, v.bit_length() - 4)
        v = v // step * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "gated", "i8"])
    if op == "norm":
        dtype = rng.choice(["bf16", "f16", "f32"])
        case = {"op": op, "rows": _size(rng, 1, 16384), "cols": _size(rng, 64, 8192),
                "dtype": dtype, "wdtype": rng.choice([dtype, "f32"]),
                "train": rng.random() < 0.6}
    elif op == "gated":
        case = {"op": op, "rows": _size(rng, 1, 4096), "hidden": _size(rng, 64, 7168),
                "cols": _size(rng, 64, 4096), "dtype": rng.choice(["bf16", "f16"]),
                "act": rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                "train": rng.random() < 0.5}
    else:
        quantise = rng.random() < 0.5
        outs = ["bf16", "f16"] if quantise else ["bf16", "f16", "f32"]
        case = {"op": op, "rows": _size(rng, 1, 8192), "n": _size(rng, 64, 8192),
                "k": _size(rng, 64, 8192), "out": rng.choice(outs), "quantise": quantise}
    return case


# ----------------------------------------------------------------- the inputs
def _draws(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=gen, device="cuda")


def _activations(randn, rows, cols):
    """A residual stream: a common offset, and a few channels much larger than
    the rest."""
    x = randn(rows, cols)
    x *= 1.0 + 7.0 * (randn(cols).abs() > 2.6)
    return x + 0.25 * randn(rows, 1)


def prepare(case, seed):
    randn = _draws(seed)
    state = {"case": case}
    if case["op"] == "norm":
        dt, wdt = DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        rows, cols = case["rows"], case["cols"]
        state["x"] = _activations(randn, rows, cols).to(dt)
        state["weight"] = (1.0 + 0.2 * randn(cols)).to(wdt)
        state["bias"] = (0.1 * randn(cols)).to(wdt)
        if case["train"]:
            state["dy"] = randn(rows, cols).to(dt)
    elif case["op"] == "gated":
        dt = DTYPES[case["dtype"]]
        rows, hidden, cols = case["rows"], case["hidden"], case["cols"]
        state["x"] = randn(rows, cols).to(dt)                 # normalised activations
        # gate rows first, then up rows
        state["weight"] = (randn(2 * hidden, cols) * cols ** -0.5).to(dt)
        if case["train"]:
            state["dh"] = randn(rows, hidden).to(dt)
    else:
        rows, n, k = case["rows"], case["n"], case["k"]
        w = randn(n, k) * k ** -0.5
        sw = w.abs().amax(1) / 127.0
        state["weight"] = torch.round(w / sw[:, None]).clamp_(-127, 127).to(torch.int8)
        state["weight_scale"] = sw
        x = _activations(randn, rows, k)
        if case["quantise"]:
            state["x"] = x.to(DTYPES[case["out"]])
        else:
            sx = x.abs().amax(1) / 127.0
            state["x"] = torch.round(x / sx[:, None]).clamp_(-127, 127).to(torch.int8)
            state["x_scale"] = sx
    return state


# ------------------------------------------------- the framework's own kernels
def _own(state):
    import dense_tiled_gemm_relu_amd as gr
    case = state["case"]
    if case["op"] == "norm":
        x, w, b = state["x"], state["weight"], state["bias"]
        if not case["train"]:
            return gr.layer_norm(x, w, b, EPS)
        y, mean, rstd = gr.layer_norm(x, w, b, EPS, stats=True)
        dx, dw, db = gr.layer_norm_backward(state["dy"], x, w, mean, rstd)
        return y, dx, dw, db
    if case["op"] == "gated":
        x, w = state["x"], state["weight"]
        if not case["train"]:
            return gr.matmul_gated(x, w, case["act"])
        h, gu = gr.matmul_gated(x, w, case["act"], save=True)
        dx, dw = gr.matmul_gated_backward(state["dh"], gu, x, w, case["act"])
        return h, dx, dw
    if case["quantise"]:
        q, s = gr.quantize_rows(state["x"])
    else:
        q, s = state["x"], state["x_scale"]
    return gr.matmul_i8(q, s, state["weight"], state["weight_scale"], DTYPES[case["out"]])


# ------------------------------------------------------------- the plain forms
def _act(g, act):
    if act == "relu":
        return torch.where(g > 0, g, torch.zeros_like(g))
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(g, act):
    if act == "relu":
        return (g > 0).to(g.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return s * (1 + g * (1 - s))
    if act == "gelu":
        return (0.5 * (1 + torch.erf(g * math.sqrt(0.5))) +
                g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi))
    t = torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 0.134145 * g * g)


def _plain(state):
    case = state["case"]
    if case["op"] == "norm":
        dt, wdt = DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        x, w, b = state["x"].float(), state["weight"].float(), state["bias"].float()
        centred = x - x.mean(1, keepdim=True)
        rstd = 1 / torch.sqrt((centred * centred).mean(1, keepdim=True) + EPS)
        xhat = centred * rstd
        y = (xhat * w + b).to(dt)
        if not case["train"]:
            return y
        dy = state["dy"].float()
        wdy = dy * w
        dx = rstd * (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True))
        return y, dx.to(dt), (dy * xhat).sum(0).to(wdt), dy.sum(0).to(wdt)
    if case["op"] == "gated":
        dt, act, hidden = DTYPES[case["dtype"]], case["act"], case["hidden"]
        x, w = state["x"].float(), state["weight"].float()
        gu = x @ w.t()
        g, u = gu[:, :hidden], gu[:, hidden:]
        a = _act(g, act)
        h = (a * u).to(dt)
        if not case["train"]:
            return h
        dh = state["dh"].float()
        dgu = torch.cat([dh * u * _act_grad(g, act), dh * a], 1)
        return h, (dgu @ w).to(dt), (dgu.t() @ x).to(dt)
    if case["quantise"]:
        x = state["x"].double()                       # values next to a rounding border
        amax = x.abs().amax(1, keepdim=True)
        q = torch.round(127 * x / amax).float()
        s = (amax[:, 0] / 127).float()
    else:
        q, s = state["x"].float(), state["x_scale"]
    y = (q @ state["weight"].float().t()) * s[:, None] * state["weight_scale"]
    return y.to(DTYPES[case["out"]])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------ the definition, 64 bits
def _phi(z):
    """The normal distribution function, from the complementary error function."""
    return 0.5 * torch.erfc(-z / math.sqrt(2.0))


def exact(case, seed):
    state = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        x, w, b = (state[k].to(f64) for k in ("x", "weight", "bias"))
        n = x.shape[1]
        mu = x.sum(1) / n
        sigma = (((x - mu[:, None]) ** 2).sum(1) / n + EPS) ** 0.5
        xhat = (x - mu[:, None]) / sigma[:, None]
        y = xhat * w + b
        if not case["train"]:
            return y
        dy = state["dy"].to(f64)
        dxhat = dy * w
        # dL/dx_j = (dxhat_j - sum_k dxhat_k (1 + xhat_j xhat_k) / n) / sigma
        s0, s1 = dxhat.sum(1), (dxhat * xhat).sum(1)
        dx = (dxhat - (s0[:, None] + xhat * s1[:, None]) / n) / sigma[:, None]
        return y, dx, (xhat * dy).sum(0), dy.sum(0)
    if case["op"] == "gated":
        act, hidden = case["act"], case["hidden"]
        x = state["x"].to(f64)
        wg, wu = state["weight"][:hidden].to(f64), state["weight"][hidden:].to(f64)
        g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
        if act == "relu":
            slope = (g > 0).to(f64)
            value = g * slope
        elif act == "silu":
            sg = torch.sigmoid(g)
            value, slope = g * sg, sg + g * sg * torch.sigmoid(-g)
        elif act == "gelu":
            value = g * _phi(g)
            slope = _phi(g) + g * torch.exp(-g * g / 2) * (2 * math.pi) ** -0.5
        else:
            # 0.5 (1 + tanh z) = sigmoid(2 z)
            c = 2 * (2 / math.pi) ** 0.5
            z = c * (g + 0.044715 * g ** 3)
            sg = torch.sigmoid(z)
            value = g * sg
            slope = sg + g * sg * torch.sigmoid(-z) * c * (1 + 3 * 0.044715 * g ** 2)
        h = value * u
        if not case["train"]:
            return h
        dh = state["dh"].to(f64)
        dg, du = dh * u * slope, dh * value
        dx = torch.mm(dg, wg) + torch.mm(du, wu)
        dw = torch.empty(2 * hidden, x.shape[1], dtype=f64, device=x.device)
        dw[:hidden] = torch.mm(dg.t(), x)
        dw[hidden:] = torch.mm(du.t(), x)
        return h, dx, dw
    wq, sw = state["weight"].to(f64), state["weight_scale"].to(f64)
    if case["quantise"]:
        x = state["x"].to(f64)
        top = x.abs().max(1).values
        q, s = torch.round(x * 127.0 / top[:, None]), top / 127.0
    else:
        q, s = state["x"].to(f64), state["x_scale"].to(f64)
    return torch.mm(q, wq.t()) * torch.outer(s, sw)


# -------------------------------------------------------- what a pass must move
def work(case):
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if case["op"] == "norm":
        e, we = size[case["dtype"]], size[case["wdtype"]]
        rows, cols = case["rows"], case["cols"]
        if case["train"]:       # x, dy in; y, dx out; the weight, the bias and their gradients
            return {"bytes": 4 * rows * cols * e + 4 * cols * we, "flops": 24 * rows * cols}
        return {"bytes": 2 * rows * cols * e + 2 * cols * we, "flops": 9 * rows * cols}
    if case["op"] == "gated":
        rows, hidden, cols = case["rows"], case["hidden"], case["cols"]
        if case["train"]:       # x, w, dh in; h, dx, dw out
            return {"bytes": 2 * (2 * rows * cols + 4 * hidden * cols + 2 * rows * hidden),
                    "flops": 12 * rows * hidden * cols}
        return {"bytes": 2 * (rows * cols + 2 * hidden * cols + rows * hidden),
                "flops": 4 * rows * hidden * cols}
    rows, n, k, out = case["rows"], case["n"], case["k"], size[case["out"]]
    x = rows * k * out if case["quantise"] else rows * k + 4 * rows
    return {"bytes": x + n * k + 4 * n + rows * n * out, "flops": 2 * rows * n * k}
