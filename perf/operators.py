"""The operators of a gated recurrent layer, as they are measured.

A layer of this kind maps its hidden rows to x | a | b, runs x through the causal conv1d + SiLU and
then through a gated linear recurrence, one state per channel:

    d_t = sigmoid(a_t),   beta_t = sigmoid(b_t),   h_t = (1 - d_t) h_{t-1} + beta_t x_t,   y_t = h_t

(1 - d_t = exp(-softplus(a_t)): the log-decay and input gate of gate_activations.) Measured are

  scan    the recurrence over packed streams, from and to carried states
  train   the recurrence and its backward pass (gradients of x, a | b and the initial states)
  step    one token for each of some streams: conv1d + SiLU on the carried window, then the recurrence
  conv    the backward pass of the causal conv1d + SiLU
  w4      the projections of a few tokens: rows times 4-bit weights with a scale for each group

Every case is a dict of plain values; `own` chooses between the plain forms below and the package.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a single user's decoding: one token through one layer, where launch latency is all there is
        dict(name="step_1", kind="step", streams=1, channels=2048, taps=4, dtype="bf16"),
        # a serving batch's decoding step
        dict(name="step_256", kind="step", streams=256, channels=4096, taps=4, dtype="bf16"),
        # a short prompt in 32 bits, not a multiple of any tile
        dict(name="scan_short_f32", kind="scan", streams=1, tokens=100, channels=768, dtype="f32"),
        # one long document: few channels, so the time axis has to be split to fill the GPU
        dict(name="scan_long", kind="scan", streams=1, tokens=65536, channels=2048, dtype="bf16"),
        # a prefill batch of prompts of very different lengths, one of them empty
        dict(name="scan_varlen", kind="scan", streams=64, tokens=262144, channels=2048, dtype="bf16"),
        # a training step on equal sequences
        dict(name="train_8x2048", kind="train", streams=8, tokens=16384, channels=4096, dtype="bf16", equal=True),
        # a training step on packed documents, odd sizes, in 32 bits
        dict(name="train_packed_f32", kind="train", streams=33, tokens=40001, channels=1000, dtype="f32"),
        # the front end's backward pass: equal sequences, the channels of 16 q, k and v heads of 128
        dict(name="conv_8x2048", kind="conv", streams=8, tokens=16384, channels=6144, taps=4, dtype="bf16", equal=True),
        # the same for packed documents, the channels of 16 q and k heads and 32 v heads
        dict(name="conv_packed", kind="conv", streams=32, tokens=100003, channels=8192, taps=4, dtype="bf16"),
        # the q | k | v | z projection of one token
        dict(name="w4_1x8192x2048", kind="w4", rows=1, outputs=8192, inputs=2048, group=128),
        # a handful of streams, an odd number of outputs, finer groups
        dict(name="w4_7x5001x4096", kind="w4", rows=7, outputs=5001, inputs=4096, group=64),
        # the widest layer and the most tokens of the range
        dict(name="w4_32x16384x8192", kind="w4", rows=32, outputs=16384, inputs=8192, group=128),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "scan", "train", "conv", "w4"])
    if kind == "w4":
        group = rng.choice([32, 64, 128])
        outputs = _log_uniform(rng, 16, 16384)
        return dict(kind=kind, rows=_log_uniform(rng, 1, 32), outputs=outputs,
                    inputs=group * max(1, _log_uniform(rng, 128, 8192) // group), group=group)
    channels = 8 * _log_uniform(rng, 8, 1024 if kind == "conv" else 512)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "step":
        return dict(kind=kind, streams=_log_uniform(rng, 1, 256), channels=channels,
                    taps=rng.randint(1, 4), dtype=dtype)
    most = {"scan": 1 << 28, "train": 1 << 25, "conv": 1 << 28}[kind] // channels
    tokens = _log_uniform(rng, 1, min(65536, most))
    case = dict(kind=kind, streams=_log_uniform(rng, 1, min(64, tokens)), tokens=tokens,
                channels=channels, dtype=dtype)
    if kind == "conv":
        case["taps"] = rng.randint(1, 4)
    return case


def work(case):
    if case["kind"] == "w4":
        m, n, k = case["rows"], case["outputs"], case["inputs"]
        return {"bytes": n * k / 2 + 2 * n * k // case["group"] + 2 * m * (k + n), "flops": 2 * m * n * k}
    e = 2 if case["dtype"] == "bf16" else 4
    B, C, K = case["streams"], case["channels"], case.get("taps", 1)
    n = case.get("tokens", B) * C
    if case["kind"] == "scan":  # x, a, b in, y out; the states both ways
        return {"bytes": 4 * e * n + 8 * B * C, "flops": 13 * n}
    if case["kind"] == "train":  # x, a, b, dy in, y, dx, da, db out; states and their gradients both ways
        return {"bytes": 8 * e * n + 16 * B * C, "flops": 36 * n}
    if case["kind"] == "step":  # x, a, b in, y out; both states both ways, the taps
        return {"bytes": 4 * e * n + 8 * n + 2 * e * (K - 1) * n + e * K * C, "flops": (18 + 2 * K) * n}
    # conv: x and dout in, dx out; the state in, its gradients in and out; taps, bias and their gradients
    return {"bytes": 3 * e * n + 3 * e * (K - 1) * B * C + (e + 4) * (K + 1) * C, "flops": (12 + 6 * K) * n}


# ------------------------------------------------------------------------------------ inputs
def _lengths(case, seed):
    """The streams' lengths: equal ones, or log-uniform over a factor of 1000 with the case's total;
    with many streams the one in the middle is empty."""
    B, T = case["streams"], case["tokens"]
    if case.get("equal"):
        return [T // B] * B
    g = torch.Generator().manual_seed(seed + 77)
    share = torch.exp(torch.rand(B, generator=g, dtype=torch.float64) * math.log(1000.0))
    if B > 8:
        share[B // 2] = 0.0
    ends = torch.round(torch.cumsum(share, 0) / share.sum() * T).to(torch.int64)
    ends[-1] = T
    return torch.diff(ends, prepend=torch.zeros(1, dtype=torch.int64)).tolist()


def _pointers(t):
    return torch.tensor([t[i].data_ptr() for i in range(t.shape[0])], dtype=torch.int64, device=DEV)


def _gates(T, C, g, dt):
    """Gate rows a | b: decay gates around a bias of each channel, so that the channels remember from
    a few to some hundreds of tokens; input gates around one half."""
    ab = torch.randn(T, 2 * C, generator=g, device=DEV)
    ab[:, :C] -= 6.0 * torch.rand(C, generator=g, device=DEV)
    return ab.to(dt)


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    if case["kind"] == "w4":
        m, n, k, group = case["rows"], case["outputs"], case["inputs"], case["group"]
        # eight weights to a 32-bit word: the even ones in the low half's nibbles, the odd ones in the high half's
        q = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        scales = ((0.5 + torch.rand(n, k // group, generator=g, device=DEV)) / (4.6 * math.sqrt(k))).to(torch.bfloat16)
        return dict(case=case, x=rand(m, k).to(torch.bfloat16), q=q, scales=scales,
                    y=torch.empty(m, n, dtype=torch.bfloat16, device=DEV))
    dt = TYPES[case["dtype"]]
    B, C, K = case["streams"], case["channels"], case.get("taps", 1)
    s = dict(case=case, B=B)
    if case["kind"] == "step":
        T = B
    else:
        T = case["tokens"]
        s["lengths"] = _lengths(case, seed)
        s["cu"] = torch.tensor([0] + s["lengths"], device=DEV).cumsum(0).to(torch.int32)
    s["x"] = rand(T, C).to(dt)
    if case["kind"] in ("scan", "train", "step"):
        s["ab"] = _gates(T, C, g, dt)
        s["h"] = rand(B, C)
        s["h_ptrs"] = _pointers(s["h"])
        s["y"] = torch.empty(T, C, dtype=dt, device=DEV)
    if case["kind"] in ("step", "conv"):
        s["w"] = (0.5 * rand(C, K)).to(dt)
        s["bias"] = (0.1 * rand(C)).to(dt)
        s["window"] = rand(B, K - 1, C).to(dt)
        s["window_ptrs"] = _pointers(s["window"]) if K > 1 else None
    if case["kind"] == "train":
        s["dy"] = rand(T, C).to(dt)
        s["dh_final"], s["dh0"] = rand(B, C), torch.empty(B, C, device=DEV)
        s["dh_final_ptrs"], s["dh0_ptrs"] = _pointers(s["dh_final"]), _pointers(s["dh0"])
        s["dx"], s["dab"] = torch.empty_like(s["x"]), torch.empty_like(s["ab"])
    if case["kind"] == "conv":
        s["dout"] = rand(T, C).to(dt)
        s["dwindow_final"], s["dwindow"] = rand(B, K - 1, C).to(dt), torch.empty(B, K - 1, C, dtype=dt, device=DEV)
        s["dwindow_final_ptrs"] = _pointers(s["dwindow_final"]) if K > 1 else None
        s["dwindow_ptrs"] = _pointers(s["dwindow"]) if K > 1 else None
        s["dx"] = torch.empty_like(s["x"])
        s["dw"], s["dbias"] = torch.empty(C, K, device=DEV), torch.empty(C, device=DEV)
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    return (_own if own else _plain)[s["case"]["kind"]](s)


def _kept(s, name, nbytes):
    """A workspace that a program keeps from call to call."""
    if name not in s:
        s[name] = torch.empty(nbytes, dtype=torch.uint8, device=DEV) if nbytes else None
    return s[name]


def _own_scan(s):
    import linear_attention_chunked_conv1d_gb300 as la
    T, C = s["x"].shape
    if "ws" not in s:
        _kept(s, "ws", la.gated_scan_workspace_bytes(s["B"], T, C, s["x"].dtype))
    la.gated_scan(s["h_ptrs"], s["x"], s["ab"], s["y"], s["cu"], workspace=s["ws"])
    return {"y": s["y"], "h": s["h"]}


def _own_train(s):
    import linear_attention_chunked_conv1d_gb300 as la
    T, C = s["x"].shape
    if "ws" not in s:
        _kept(s, "ws", la.gated_scan_workspace_bytes(s["B"], T, C, s["x"].dtype))
        _kept(s, "saved", la.gated_scan_saved_bytes(s["B"], T, C, s["x"].dtype))
    la.gated_scan(s["h_ptrs"], s["x"], s["ab"], s["y"], s["cu"], saved=s["saved"], workspace=s["ws"])
    la.gated_scan_backward(s["x"], s["ab"], s["saved"], s["dy"], s["dx"], s["dab"], s["cu"],
                           dh_final_ptrs=s["dh_final_ptrs"], dh0_ptrs=s["dh0_ptrs"], workspace=s["ws"])
    return {"y": s["y"], "h": s["h"], "dx": s["dx"], "dab": s["dab"], "dh0": s["dh0"]}


def _own_step(s):
    import linear_attention_chunked_conv1d_gb300 as la
    la.gated_scan_step(s["h_ptrs"], s["x"], s["ab"], s["y"], conv_state_ptrs=s["window_ptrs"], conv_w=s["w"],
                       conv_bias=s["bias"])
    return {"y": s["y"], "h": s["h"], "window": s["window"]}


def _own_conv(s):
    import linear_attention_chunked_conv1d_gb300 as la
    T, C = s["x"].shape
    if "ws" not in s:
        _kept(s, "ws", la.conv1d_silu_backward_workspace_bytes(s["B"], T, C, s["w"].shape[1], s["x"].dtype))
    la.conv1d_silu_backward(s["window_ptrs"], s["x"], s["w"], s["dout"], s["dx"], s["dw"], s["cu"], bias=s["bias"],
                            dbias=s["dbias"], dstate_final_ptrs=s["dwindow_final_ptrs"], dstate_ptrs=s["dwindow_ptrs"],
                            workspace=s["ws"])
    return {"dx": s["dx"], "dw": s["dw"], "dbias": s["dbias"], "dwindow": s["dwindow"]}


def _own_w4(s):
    import linear_attention_chunked_conv1d_gb300 as la
    return {"y": la.w4_matvec(s["x"], s["q"], s["scales"], s["y"])}


_own = {"scan": _own_scan, "train": _own_train, "step": _own_step, "conv": _own_conv, "w4": _own_w4}


def _joined(keep, add, longest):
    """h_t = keep_t h_{t-1} + add_t along the rows (keep is zero where a stream starts): runs of rows are
    joined in pairs, each time of twice the length."""
    n = 1
    while n < longest:
        add[n:] = add[n:] + keep[n:] * add[:-n]
        keep[n:] = keep[n:] * keep[:-n]
        n *= 2
    return add


def _plain_forward(s):
    C = s["x"].shape[1]
    keep, beta = torch.sigmoid(-s["ab"][:, :C].float()), torch.sigmoid(s["ab"][:, C:].float())
    first, last = s["cu"][:-1].long(), s["cu"][1:].long() - 1
    full = last >= first
    add = beta * s["x"].float()
    add[first[full]] += keep[first[full]] * s["h"][full]
    keep[first[full]] = 0
    h = _joined(keep, add, max(s["lengths"]))
    return h, first[full], last[full], full


def _plain_scan(s):
    h, _, last, full = _plain_forward(s)
    s["h"][full] = h[last]
    return {"y": h.to(s["x"].dtype), "h": s["h"]}


def _plain_train(s):
    C, dt = s["x"].shape[1], s["x"].dtype
    h0 = s["h"].clone()
    h, first, last, full = _plain_forward(s)
    s["h"][full] = h[last]
    y = h.to(dt)
    before = torch.cat([h[:1], h[:-1]])
    before[first] = h0[full]
    a, b = s["ab"][:, :C].float(), s["ab"][:, C:].float()
    keep, d, beta = torch.sigmoid(-a), torch.sigmoid(a), torch.sigmoid(b)
    # the gradient of h_t: dy_t, and what the next token of the stream keeps of it
    grad = s["dy"].float().clone()
    grad[last] += s["dh_final"][full]
    after = torch.cat([keep[1:], keep[:1]])
    after[last] = 0
    grad = _joined(after.flip(0), grad.flip(0), max(s["lengths"])).flip(0)
    dh0 = s["dh_final"].clone()
    dh0[full] = (keep * grad)[first]
    s["dh0"].copy_(dh0)
    dab = torch.cat([-grad * before * keep * d, grad * s["x"].float() * beta * (1 - beta)], 1)
    return {"y": y, "h": s["h"], "dx": (grad * beta).to(dt), "dab": dab.to(dt), "dh0": s["dh0"]}


def _plain_step(s):
    C, K = s["w"].shape
    rows = torch.cat([s["window"].float(), s["x"].float()[:, None]], 1)  # [B][K][C], oldest first
    p = (rows * s["w"].float().t()).sum(1) + s["bias"].float()
    x = p * torch.sigmoid(p)
    a, b = s["ab"][:, :C].float(), s["ab"][:, C:].float()
    h = torch.sigmoid(-a) * s["h"] + torch.sigmoid(b) * x
    s["h"].copy_(h)
    s["window"].copy_(rows[:, 1:])
    return {"y": h.to(s["x"].dtype), "h": s["h"], "window": s["window"]}


def _plain_conv(s):
    C, K = s["w"].shape
    T, dt, cu = s["x"].shape[0], s["x"].dtype, s["cu"].long()
    first, length = cu[:-1], cu[1:] - cu[:-1]
    stream = torch.repeat_interleave(torch.arange(s["B"], device=DEV), length)
    place = torch.arange(T, device=DEV) - first[stream]  # of a token in its stream
    x, w = s["x"].float(), s["w"].float()

    def back(n):
        """The row n before each token: one of its stream, or of the window that the stream came with."""
        early = place < n
        rows = torch.cat([x[:1].expand(n, C), x])[:T]
        rows[early] = s["window"][stream[early], place[early] - n + K - 1].float()
        return rows

    p = s["bias"].float().expand(T, C).clone()
    for j in range(K):
        p += w[:, j] * back(K - 1 - j)
    sig = torch.sigmoid(p)
    dp = s["dout"].float() * sig * (1 + p * (1 - sig))
    dw = torch.stack([(dp * back(K - 1 - j)).sum(0, dtype=torch.float64) for j in range(K)], 1)
    dx = torch.zeros(T, C, device=DEV)
    dwindow = torch.zeros(s["B"], K - 1, C, device=DEV)
    for n in range(K):  # dp of a token goes to the row n before it
        inside = place >= n
        if n < T:
            dx[:T - n] += torch.where(inside[n:, None], w[:, K - 1 - n] * dp[n:], 0.0)
        if n:
            at = (~inside).nonzero()[:, 0]
            dwindow.index_put_((stream[at], place[at] - n + K - 1), w[:, K - 1 - n] * dp[at], accumulate=True)
    for m in range(K - 1):  # row m of the window that the stream leaves: its row length + m of window | tokens
        row = length + m - (K - 1)
        dx[first[row >= 0] + row[row >= 0]] += s["dwindow_final"][row >= 0, m].float()
        at = (row < 0).nonzero()[:, 0]
        dwindow.index_put_((at, row[at] + K - 1), s["dwindow_final"][at, m].float(), accumulate=True)
    s["dwindow"].copy_(dwindow)
    return {"dx": dx.to(dt), "dw": dw.float(), "dbias": dp.sum(0, dtype=torch.float64).float(), "dwindow": s["dwindow"]}


def _plain_w4(s):
    n, k = s["q"].shape[0], s["q"].shape[1] * 2
    q = s["q"].view(n, k // 8, 4).to(torch.int32)
    word = q[..., 0] | q[..., 1] << 8 | q[..., 2] << 16 | q[..., 3] << 24
    at = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=DEV, dtype=torch.int32)
    w = ((word[..., None] >> at) & 15).view(n, -1, s["case"]["group"]).float() - 8.0
    w = (w * s["scales"].float()[..., None]).view(n, k)
    return {"y": (s["x"].float() @ w.t()).to(torch.bfloat16)}


_plain = {"scan": _plain_scan, "train": _plain_train, "step": _plain_step, "conv": _plain_conv, "w4": _plain_w4}


# ------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_scan, "train": _exact_scan, "step": _exact_step, "conv": _exact_conv, "w4": _exact_w4}[case["kind"]](s)


def _exact_scan(s):
    """Token after token, all streams side by side."""
    train = s["case"]["kind"] == "train"
    longest = max(s["lengths"])
    if longest > (50000 if train else 150000):
        return None
    (T, C), B = s["x"].shape, s["B"]
    a, b, x = s["ab"][:, :C].double(), s["ab"][:, C:].double(), s["x"].double()
    keep, beta = 1 / (1 + torch.exp(a)), 1 / (1 + torch.exp(-b))
    h = s["h"].double()
    y, old = torch.empty_like(x), torch.empty_like(x) if train else None
    # streams in order of length, so that those still running are the first ones
    order = sorted(range(B), key=lambda i: -s["lengths"][i])
    start = s["cu"].long()[:-1][torch.tensor(order, device=DEV)]
    now, length = h[torch.tensor(order, device=DEV)], [s["lengths"][i] for i in order]
    running = [0] * (longest + 1)
    n = B
    for t in range(longest):
        while length[n - 1] <= t:
            n -= 1
        running[t] = n
        at = start[:n] + t
        if train:
            old[at] = now[:n]
        now[:n] = keep[at] * now[:n] + beta[at] * x[at]
        y[at] = now[:n]
    h[torch.tensor(order, device=DEV)] = now
    if not train:
        return {"y": y, "h": h}
    dy, grad = s["dy"].double(), torch.empty_like(x)
    back = s["dh_final"].double()[torch.tensor(order, device=DEV)]
    for t in range(longest - 1, -1, -1):
        n = running[t]
        at = start[:n] + t
        grad[at] = dy[at] + back[:n]
        back[:n] = keep[at] * grad[at]
    dh0 = torch.empty_like(back)
    dh0[torch.tensor(order, device=DEV)] = back
    da = -grad * old * keep * (1 - keep)
    return {"y": y, "h": h, "dx": grad * beta, "dab": torch.cat([da, grad * x * beta * (1 - beta)], 1), "dh0": dh0}


def _exact_step(s):
    C, K = s["w"].shape
    p = s["bias"].double() + s["x"].double() * s["w"][:, K - 1].double()
    for j in range(K - 1):
        p = p + s["window"][:, j].double() * s["w"][:, j].double()
    x = p / (1 + torch.exp(-p))
    d, beta = 1 / (1 + torch.exp(-s["ab"][:, :C].double())), 1 / (1 + torch.exp(-s["ab"][:, C:].double()))
    h = s["h"].double() * (1 - d) + beta * x
    return {"y": h, "h": h, "window": torch.cat([s["window"][:, 1:], s["x"][:, None]], 1).double() if K > 1 else s["window"].double()}


def _exact_conv(s):
    """Differentiated stream by stream, with the convolution as torch has it."""
    K, B = s["w"].shape[1], s["B"]
    w, bias = (s[n].double().requires_grad_() for n in ("w", "bias"))
    dx, dwindow, total = [], [], [torch.zeros_like(w), torch.zeros_like(bias)]
    ends = s["cu"].tolist()
    for i in range(B):
        x = s["x"][ends[i]:ends[i + 1]].double().requires_grad_()
        window = s["window"][i].double().requires_grad_()
        rows = torch.cat([window, x])
        left, grads = [rows[rows.shape[0] - (K - 1):]], [s["dwindow_final"][i].double()]
        if x.shape[0]:
            p = torch.nn.functional.conv1d(rows.t()[None], w[:, None], bias, groups=w.shape[0])[0].t()
            left, grads = left + [p / (1 + torch.exp(-p))], grads + [s["dout"][ends[i]:ends[i + 1]].double()]
        g = torch.autograd.grad(left, (x, window, w, bias), grads, allow_unused=True)
        g = [torch.zeros_like(v) if u is None else u for u, v in zip(g, (x, window, w, bias))]
        dx.append(g[0]), dwindow.append(g[1])
        total = [total[0] + g[2], total[1] + g[3]]
    return {"dx": torch.cat(dx), "dw": total[0], "dbias": total[1], "dwindow": torch.stack(dwindow)}


def _exact_w4(s):
    n, k, group = s["q"].shape[0], s["q"].shape[1] * 2, s["case"]["group"]
    w = torch.empty(n, k // 8, 8, dtype=torch.float64, device=DEV)
    byte = s["q"].view(n, k // 8, 4)
    for i in range(4):  # weight 2i: nibble i of the word; weight 2i + 1: nibble i + 4
        low = byte[..., i // 2]
        high = byte[..., 2 + i // 2]
        w[..., 2 * i] = (low >> 4 if i % 2 else low & 15).double() - 8
        w[..., 2 * i + 1] = (high >> 4 if i % 2 else high & 15).double() - 8
    w = w.view(n, k) * s["scales"].double().repeat_interleave(group, 1)
    return {"y": s["x"].double() @ w.t()}
