"""The operators of a layer's dense half, as they are measured.

Next to the recurrent half of a layer stand a norm of the hidden rows, a gated feed-forward block
and products with bias, activation and residual in their epilogue:

    norm    y = (x - mean(x)) / sqrt(var(x) + eps) * w + b, one row at a time
    linear  y = act(x W^T + bias) + residual
    ffn     h = act(x Wg^T) * (x Wu^T): gate and up projection, activation and product

Each is measured as a forward call and, with train=True, as the forward and the backward pass of a
training step (gradients of the inputs, the weights and the biases). Activations `act` are "none",
"relu", "gelu" (with the normal distribution's integral), "gelu_tanh" and "silu".

Every case is a dict of plain values; `own` chooses between the plain forms below and the package.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a single user's decoding: the norm of one token, where launch latency is all there is
        dict(name="norm_1x2048", kind="norm", rows=1, width=2048, dtype="bf16", train=False),
        # a training step on a batch of sequences, with the gradient that passes the layer by
        dict(name="norm_train_16384x4096", kind="norm", rows=16384, width=4096, dtype="bf16", train=True, skip=True),
        # a training step in 32 bits, an odd number of rows, a width that no vector divides
        dict(name="norm_train_f32_5001x1001", kind="norm", rows=5001, width=1001, dtype="f32", train=True, skip=False),
        # decoding: one token through the projection q | k | v | z, with a bias
        dict(name="linear_1x8192x2048", kind="linear", rows=1, outputs=8192, inputs=2048, act="none", bias=True, residual=False, train=False),
        # a short prompt, an odd number of outputs, activation and residual
        dict(name="linear_777x5001x2048", kind="linear", rows=777, outputs=5001, inputs=2048, act="gelu", bias=True, residual=True, train=False),
        # prefill: the projection back to the hidden rows, onto the residual stream
        dict(name="linear_16384x4096x8192", kind="linear", rows=16384, outputs=4096, inputs=8192, act="none", bias=False, residual=True, train=False),
        # a training step of a feed-forward block without a gate
        dict(name="linear_train_8192x8192x2048", kind="linear", rows=8192, outputs=8192, inputs=2048, act="gelu_tanh", bias=True, residual=False, train=True),
        # decoding: one token
        dict(name="ffn_1x8192x2048", kind="ffn", rows=1, hidden=8192, inputs=2048, act="silu", train=False),
        # decoding: a serving batch
        dict(name="ffn_32x8192x4096", kind="ffn", rows=32, hidden=8192, inputs=4096, act="silu", train=False),
        # prefill of many prompts
        dict(name="ffn_16384x8192x4096", kind="ffn", rows=16384, hidden=8192, inputs=4096, act="silu", train=False),
        # a training step on equal sequences
        dict(name="ffn_train_8192x8192x4096", kind="ffn", rows=8192, hidden=8192, inputs=4096, act="silu", train=True),
        # a training step on packed documents, odd sizes
        dict(name="ffn_train_4099x2733x1000", kind="ffn", rows=4099, hidden=2733, inputs=1000, act="gelu", train=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "linear", "ffn"])
    train = rng.random() < 0.5
    if kind == "norm":
        width = _log_uniform(rng, 64, 8192)
        return dict(kind=kind, rows=_log_uniform(rng, 1, min(65536, (1 << 26) // width)), width=width,
                    dtype=rng.choice(["bf16", "f32"]), train=train, skip=train and rng.random() < 0.5)
    inputs, outputs = _log_uniform(rng, 64, 8192), _log_uniform(rng, 64, 8192)
    # no dearer than the largest listed case: 3.3 TFLOP of a training step through the gated block
    per_row = (3 if train else 1) * (4 if kind == "ffn" else 2) * inputs * outputs
    rows = _log_uniform(rng, 1, max(1, min(16384, int(3.0e12) // per_row)))
    if kind == "ffn":
        return dict(kind=kind, rows=rows, hidden=outputs, inputs=inputs, act=rng.choice(["silu", "gelu", "gelu_tanh"]), train=train)
    # relu's derivative jumps at 0, so a training step with it has no value there to compare
    return dict(kind=kind, rows=rows, outputs=outputs, inputs=inputs, act=rng.choice(["none", "gelu", "gelu_tanh", "silu"] + ([] if train else ["relu"])),
                bias=rng.random() < 0.5, residual=rng.random() < 0.5, train=train)


def work(case):
    m = case["rows"]
    if case["kind"] == "norm":
        n, e, d = case["width"], 2 if case["dtype"] == "bf16" else 4, case["train"]
        # x in, y out, w and b; in training dy in, dx out, the gradient that passes by, w's and b's gradients
        return {"bytes": e * m * n * (2 + (2 + case.get("skip", False) if d else 0)) + 2 * e * n + (8 * n if d else 0),
                "flops": (20 if d else 8) * m * n}
    n, k = case["outputs"] if case["kind"] == "linear" else case["hidden"], case["inputs"]
    if case["kind"] == "linear":
        # x, W, bias, residual in, y out; in training dy in, the gradients of x, W and the bias out
        nbytes = 2 * (m * k + n * k + m * n * (1 + case["residual"]) + n * case["bias"])
        return {"bytes": nbytes + (2 * (m * n + m * k + n * k + n * case["bias"]) if case["train"] else 0),
                "flops": (6 if case["train"] else 2) * m * n * k}
    # x and both weights in, h out; in training dh in, the gradients of x and both weights out
    nbytes = 2 * (m * k + 2 * n * k + m * n)
    return {"bytes": nbytes * (2 if case["train"] else 1), "flops": (12 if case["train"] else 4) * m * n * k}


# ------------------------------------------------------------------------------------ inputs
def _rows(t, rows, cols, g=None, std=1.0):
    """A matrix whose rows start on 16 bytes, as a program with an odd number of columns keeps it; normal
    values, or uninitialised without g."""
    per = 16 // t.itemsize
    ld = (cols + per - 1) // per * per
    if g is None:
        return torch.empty(rows, ld, dtype=t, device=DEV)[:, :cols]
    return torch.randn(rows, ld, generator=g, device=DEV).mul_(std).to(t)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    m, bf16 = case["rows"], torch.bfloat16
    s = dict(case=case)
    if case["kind"] == "norm":
        n, dt = case["width"], TYPES[case["dtype"]]
        x = _rows(torch.float32, m, n, g)
        # hidden rows: channels of different sizes, a few of them large, a mean of its own to each row
        x = x * (0.5 + torch.rand(n, generator=g, device=DEV)) + 0.3 * torch.randn(m, 1, generator=g, device=DEV)
        x[:, torch.randint(0, n, (max(1, n // 512),), generator=g, device=DEV)] *= 12.0
        s["x"], s["y"] = _rows(dt, m, n), _rows(dt, m, n)
        s["x"].copy_(x)
        s["w"] = (1.0 + 0.2 * torch.randn(n, generator=g, device=DEV)).to(dt)
        s["b"] = (0.1 * torch.randn(n, generator=g, device=DEV)).to(dt)
        if case["train"]:
            s["dy"], s["dx"] = _rows(dt, m, n, g), _rows(dt, m, n)
            s["dskip"] = _rows(dt, m, n, g) if case.get("skip") else None
            s["stats"] = torch.empty(m, 2, device=DEV)
            s["dw"], s["db"] = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
        return s
    n, k = case["outputs"] if case["kind"] == "linear" else case["hidden"], case["inputs"]
    s["x"], s["y"] = _rows(bf16, m, k, g), _rows(bf16, m, n)
    if case["kind"] == "linear":
        s["w"] = _rows(bf16, n, k, g, 1.0 / math.sqrt(k))
        s["bias"] = (0.3 * torch.randn(n, generator=g, device=DEV)).to(bf16) if case["bias"] else None
        s["residual"] = _rows(bf16, m, n, g) if case["residual"] else None
    else:
        s["w_gate"], s["w_up"] = _rows(bf16, n, k, g, 1.0 / math.sqrt(k)), _rows(bf16, n, k, g, 1.0 / math.sqrt(k))
    if case["train"]:
        s["dy"], s["dx"] = _rows(bf16, m, n, g), _rows(bf16, m, k)
        if case["kind"] == "linear":
            s["dw"] = _rows(bf16, n, k)
            s["dbias"] = torch.empty(n, dtype=bf16, device=DEV) if case["bias"] else None
        else:
            s["dw_gate"], s["dw_up"] = _rows(bf16, n, k), _rows(bf16, n, k)
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)[s["case"]["kind"]](s)


def _kept(s, name, nbytes):
    """A buffer that a program keeps from call to call."""
    if name not in s:
        s[name] = torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None
    return s[name]


def _own_norm(s):
    import linear_attention_chunked_conv1d_gb300 as la
    if not s["case"]["train"]:
        return {"y": la.layernorm_rows(s["x"], s["w"], s["b"], s["y"], eps=EPS)}
    la.layernorm_rows(s["x"], s["w"], s["b"], s["y"], eps=EPS, stats=s["stats"])
    if "ws" not in s:
        _kept(s, "ws", la.layernorm_rows_backward_workspace_bytes(*s["x"].shape, s["x"].dtype))
    la.layernorm_rows_backward(s["x"], s["w"], s["stats"], s["dy"], s["dx"], s["dw"], s["db"], dskip=s["dskip"], workspace=s["ws"])
    return {"y": s["y"], "dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def _own_linear(s):
    import linear_attention_chunked_conv1d_gb300 as la
    act, train = s["case"]["act"], s["case"]["train"]
    (m, k), n = s["x"].shape, s["w"].shape[0]
    if train and "ws" not in s:
        _kept(s, "ws", la.linear_backward_workspace_bytes(m, n, k, act))
        _kept(s, "saved", la.linear_saved_bytes(m, n, act))
    la.linear(s["x"], s["w"], s["y"], bias=s["bias"], residual=s["residual"], act=act, saved=s["saved"] if train else None)
    if not train:
        return {"y": s["y"]}
    la.linear_backward(s["x"], s["w"], s["saved"], s["dy"], s["dx"], s["dw"], dbias=s["dbias"], act=act, workspace=s["ws"])
    out = {"y": s["y"], "dx": s["dx"], "dw": s["dw"]}
    return out | {"dbias": s["dbias"]} if s["dbias"] is not None else out


def _own_ffn(s):
    import linear_attention_chunked_conv1d_gb300 as la
    act, train = s["case"]["act"], s["case"]["train"]
    (m, k), n = s["x"].shape, s["w_gate"].shape[0]
    if train and "ws" not in s:
        _kept(s, "ws", la.gated_ffn_backward_workspace_bytes(m, n, k))
        _kept(s, "saved", la.gated_ffn_saved_bytes(m, n))
    la.gated_ffn(s["x"], s["w_gate"], s["w_up"], s["y"], act=act, saved=s["saved"] if train else None)
    if not train:
        return {"y": s["y"]}
    la.gated_ffn_backward(s["x"], s["w_gate"], s["w_up"], s["saved"], s["dy"], s["dx"], s["dw_gate"], s["dw_up"], act=act, workspace=s["ws"])
    return {"y": s["y"], "dx": s["dx"], "dw_gate": s["dw_gate"], "dw_up": s["dw_up"]}


_own = {"norm": _own_norm, "linear": _own_linear, "ffn": _own_ffn}


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.clamp_min(z, 0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))


def _act_slope(z, act):
    """The derivative of the activation (a factor for the gradient)."""
    if act == "none":
        return 1.0
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))


def _plain_norm(s):
    dt = s["x"].dtype
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    c = x - x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    xh = c * rstd
    y = (xh * w + b).to(dt)
    if not s["case"]["train"]:
        return {"y": y}
    dy = s["dy"].float()
    dxh = dy * w
    dx = rstd * (dxh - dxh.mean(1, keepdim=True) - xh * (dxh * xh).mean(1, keepdim=True))
    if s["dskip"] is not None:
        dx = dx + s["dskip"].float()
    return {"y": y, "dx": dx.to(dt), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def _plain_linear(s):
    act, bf16 = s["case"]["act"], torch.bfloat16
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, act)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(bf16)}
    if s["case"]["train"]:
        dz = s["dy"].float() * _act_slope(z, act)
        out |= {"dx": (dz @ w).to(bf16), "dw": (dz.T @ x).to(bf16)}
        if s["bias"] is not None:
            out["dbias"] = dz.sum(0).to(bf16)
    return out


def _plain_ffn(s):
    act, bf16 = s["case"]["act"], torch.bfloat16
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    gate, up = x @ wg.T, x @ wu.T
    a = _act(gate, act)
    out = {"y": (a * up).to(bf16)}
    if s["case"]["train"]:
        dh = s["dy"].float()
        dgate, dup = dh * up * _act_slope(gate, act), dh * a
        out |= {"dx": (dgate @ wg + dup @ wu).to(bf16), "dw_gate": (dgate.T @ x).to(bf16), "dw_up": (dup.T @ x).to(bf16)}
    return out


_plain = {"norm": _plain_norm, "linear": _plain_linear, "ffn": _plain_ffn}


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The outputs in 64 bits, from the definitions; gradients by torch's own differentiation."""
    s = prepare(case, seed)
    kind, train = case["kind"], case["train"]
    x = s["x"].double().requires_grad_(train)
    if kind == "norm":
        weights = [s["w"].double().requires_grad_(train), s["b"].double().requires_grad_(train)]
        var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
        y = (x - mean) * torch.rsqrt(var + EPS) * weights[0] + weights[1]
        names = ["dw", "db"]
    elif kind == "linear":
        weights = [s["w"].double().requires_grad_(train)]
        names = ["dw"]
        y = torch.nn.functional.linear(x, weights[0])
        if s["bias"] is not None:
            weights.append(s["bias"].double().requires_grad_(train))
            names.append("dbias")
            y = y + weights[1]
        y = _exact_act(y, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].double()
    else:
        weights = [s["w_gate"].double().requires_grad_(train), s["w_up"].double().requires_grad_(train)]
        y = _exact_act(torch.nn.functional.linear(x, weights[0]), case["act"]) * torch.nn.functional.linear(x, weights[1])
        names = ["dw_gate", "dw_up"]
    out = {"y": y.detach()}
    if train:
        grads = torch.autograd.grad(y, [x] + weights, s["dy"].double())
        out["dx"] = grads[0]
        if s.get("dskip") is not None:
            out["dx"] = out["dx"] + s["dskip"].double()
        out |= dict(zip(names, grads[1:]))
    return out


def _exact_act(z, act):
    F = torch.nn.functional
    if act == "none":
        return z
    return {"relu": F.relu, "silu": F.silu, "gelu": F.gelu, "gelu_tanh": lambda t: F.gelu(t, approximate="tanh")}[act](z)
