"""The gated recurrence (scan, backward pass, decode step) on the GPU against a plain token-by-token
form in 64 bits, with a running bound of the rounding errors of 32-bit arithmetic.

Bounds, for gates |a|, |b| <= 8: a gate is 1 / (1 + 2^(-a log2 e)); the argument's rounding moves the
exponential by at most 8 * 2^-24 relative to it, the hardware exponential and reciprocal and four more
roundings add less than 2^-22 + 2^-23 + 4 * 2^-24, in all EPS = 2^-20 is never reached. A token adds
EPS (d |h| + beta |x|) for its gates and, with the roundings of the update itself and of the joins of
runs of tokens, less than 4 * 2^-24 (|h| + beta |x|); what is there already decays with 1 - d. The sums
of the backward pass have the same form. A result in bf16 is off by half a step of its own more.
"""
import numpy as np
import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la
from tests.helpers import f64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS, UPDATE = 2.0 ** -20, 2.0 ** -22


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def forward(x, a, b, h0, lengths):
    """y, states before each token, final states, and the bound of y's (and the states') errors."""
    y, before, err, err_before = (np.zeros_like(x) for _ in range(4))
    final, t = h0.copy(), 0
    final_err = np.zeros_like(h0)
    d, beta = sigmoid(a), sigmoid(b)
    for s, n in enumerate(lengths):
        h, e = h0[s].copy(), np.zeros(x.shape[1])
        for t in range(t, t + n):
            before[t], err_before[t] = h, e
            u = beta[t] * x[t]
            e = (1 - d[t]) * e + EPS * (d[t] * abs(h) + abs(u)) + UPDATE * (abs(h) + abs(u))
            h = (1 - d[t]) * h + u
            y[t], err[t] = h, e
        t += n > 0
        final[s], final_err[s] = h, e
    return y, before, final, err, err_before, final_err


def backward(x, a, b, before, err_before, dy, dfinal, lengths):
    d, beta = sigmoid(a), sigmoid(b)
    lam, err = np.zeros_like(x), np.zeros_like(x)
    dh0, dh0_err = dfinal.copy(), np.zeros_like(dfinal)
    end = sum(lengths)
    for s in reversed(range(len(lengths))):
        m, e = dfinal[s].copy(), np.zeros(x.shape[1])
        for t in range(end - 1, end - 1 - lengths[s], -1):
            lam[t] = dy[t] + m
            err[t] = e + UPDATE * (abs(dy[t]) + abs(m))
            m = (1 - d[t]) * lam[t]
            e = (1 - d[t]) * err[t] + (EPS * d[t] + UPDATE) * abs(lam[t])
        end -= lengths[s]
        dh0[s], dh0_err[s] = m, e
    dx = lam * beta
    db = dx * x * (1 - beta)
    da = -lam * before * d * (1 - d)
    # three factors of one gate, and the error of 1 - gate relative to the gate's own
    gate = 4 * EPS
    dx_err = err * beta + EPS * abs(dx)
    db_err = err * abs(x) * beta * (1 - beta) + gate * abs(lam * x) * beta
    da_err = (err * abs(before) + abs(lam) * err_before) * d * (1 - d) + gate * abs(lam * before) * d
    return (dx, dx_err), (np.concatenate([da, db], 1), np.concatenate([da_err, db_err], 1)), (dh0, dh0_err)


def close(got, want, err, dtype="f32"):
    got = f64(got)
    tol = 2 * err + HALF[dtype] * (abs(want) + 2 * err) + 1e-37
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - want) / tol) if got.size else 0.0
    assert worst <= 1, worst


def make(lengths, C, dtype, seed, slow=0.0):
    g = torch.Generator().manual_seed(seed)
    T, B = sum(lengths), len(lengths)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    ab = r(T, 2 * C)
    ab[:, :C] -= slow * torch.rand(C, generator=g)
    return dict(x=r(T, C).to(DT[dtype]), ab=ab.clamp(-8, 8).to(DT[dtype]), h=r(B, C), dy=r(T, C).to(DT[dtype]),
                dfinal=r(B, C))


def cu_of(lengths, dev):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=dev)


def workspace(fn, *args, dev):
    return torch.empty(fn(*args), dtype=torch.uint8, device=dev).fill_(0xA5)


def gpu_pass(cuda, inp, lengths, *, packed=True, states=True, grads=True):
    """Forward with saved states, then backward, on the GPU; every output pre-filled."""
    T, C = inp["x"].shape
    B, dt = len(lengths), inp["x"].dtype
    x, ab, dy = (inp[n].to(cuda) for n in ("x", "ab", "dy"))
    h, dfin = inp["h"].clone().to(cuda), inp["dfinal"].to(cuda)
    dh0 = torch.full_like(dfin, 9.0)
    y, dx, dab = (torch.full_like(v, 7.0) for v in (x, x, ab))
    cu = cu_of(lengths, cuda) if packed else None
    ws = workspace(la.gated_scan_workspace_bytes, B, T, C, dt, dev=cuda)
    saved = workspace(la.gated_scan_saved_bytes, B, T, C, dt, dev=cuda)
    la.gated_scan(la.pointer_array(list(h)) if states else None, x, ab, y, cu, B=B, saved=saved, workspace=ws)
    la.gated_scan_backward(x, ab, saved, dy, dx, dab, cu, B=B, workspace=ws,
                           dh_final_ptrs=la.pointer_array(list(dfin)) if grads else None,
                           dh0_ptrs=la.pointer_array(list(dh0)) if grads else None)
    torch.cuda.synchronize()
    assert la.device_status() == 0
    return y, h, dx, dab, dh0


LENGTHS = {
    "empty first": [0, 0, 5], "between the tiles": [0, 150, 0, 1, 100], "a tile": [100, 156], "over a tile": [100, 157],
    "one": [1], "two": [2], "short": [37], "tile": [64], "tile+1": [65], "batch": [100, 100, 100],
    "ones": [1] * 70, "ragged": [0, 1, 63, 64, 65, 0, 0, 130, 7, 0], "long": [5000], "mixed": [3, 1900, 0, 1, 700, 64],
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [8, 136, 520])
@pytest.mark.parametrize("name", LENGTHS)
def test_forward_and_backward(cuda, name, C, dtype):
    lengths = LENGTHS[name]
    inp = make(lengths, C, dtype, seed=C + len(name), slow=6.0)
    x, ab, dy = (f64(inp[n]) for n in ("x", "ab", "dy"))
    a, b = ab[:, :C], ab[:, C:]
    y_r, before, fin, err, err_b, fin_err = forward(x, a, b, f64(inp["h"]), lengths)
    dx_r, dab_r, dh0_r = backward(x, a, b, before, err_b, dy, f64(inp["dfinal"]), lengths)
    y, h, dx, dab, dh0 = gpu_pass(cuda, inp, lengths, packed=name != "batch")
    close(y, y_r, err, dtype)
    close(h, fin, fin_err)
    close(dx, *dx_r, dtype)
    close(dab, *dab_r, dtype)
    close(dh0, *dh0_r)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_without_states_and_state_gradients(cuda, dtype):
    lengths, C = [90, 0, 300], 72
    inp = make(lengths, C, dtype, seed=5)
    zero = np.zeros((3, C))
    x, ab, dy = (f64(inp[n]) for n in ("x", "ab", "dy"))
    y_r, before, _, err, err_b, _ = forward(x, ab[:, :C], ab[:, C:], zero, lengths)
    dx_r, dab_r, _ = backward(x, ab[:, :C], ab[:, C:], before, err_b, dy, zero, lengths)
    y, h, dx, dab, dh0 = gpu_pass(cuda, inp, lengths, states=False, grads=False)
    close(y, y_r, err, dtype)
    close(dx, *dx_r, dtype)
    close(dab, *dab_r, dtype)
    assert torch.equal(h.cpu(), inp["h"]) and torch.all(dh0 == 9.0)


def test_gradients_against_differences(cuda):
    """Central differences of the 64-bit form's own loss, at a few places of every input: the formula
    of the gradients is the function's (the plain form above shares it with the kernels)."""
    lengths, C = [5, 0, 9], 8
    inp = make(lengths, C, "f32", seed=6)
    v = {"x": f64(inp["x"]), "ab": f64(inp["ab"]), "h": f64(inp["h"])}
    dy, dfin = f64(inp["dy"]), f64(inp["dfinal"])

    def loss(v):
        y, _, fin, *_ = forward(v["x"], v["ab"][:, :C], v["ab"][:, C:], v["h"], lengths)
        return (y * dy).sum() + (fin * dfin).sum()

    _, _, dx, dab, dh0 = gpu_pass(cuda, inp, lengths)
    step = 1e-5
    for name, got in (("x", dx), ("ab", dab), ("h", dh0)):
        got = f64(got)
        for i in np.ndindex(got.shape):
            up, down = ({k: u.copy() for k, u in v.items()} for _ in range(2))
            up[name][i] += step
            down[name][i] -= step
            want = (loss(up) - loss(down)) / (2 * step)
            # the kernel: up to four gate errors, relative to products that pass the gradient itself by
            # 1 / (1 - gate) at most; the differences: under 1e-7 (step^2, and 1e-15 * 100 / step)
            assert abs(got[i] - want) <= 8 * EPS * (1 + abs(want)), (name, i)


def test_split_calls_carry_the_state(cuda):
    """A sequence in two calls gives the whole's y; the tile grid starts anew, so not bit for bit."""
    T, C, cut = 700, 64, 333
    inp = make([T], C, "f32", seed=7, slow=6.0)
    y_r, _, fin, err, _, fin_err = forward(f64(inp["x"]), f64(inp["ab"])[:, :C], f64(inp["ab"])[:, C:], f64(inp["h"]), [T])
    x, ab, h = (inp[n].clone().to(cuda) for n in ("x", "ab", "h"))
    y = torch.empty_like(x)
    ws = workspace(la.gated_scan_workspace_bytes, 1, T, C, x.dtype, dev=cuda)
    ptrs = la.pointer_array(list(h))
    for lo, hi in ((0, cut), (cut, T)):
        la.gated_scan(ptrs, x[lo:hi], ab[lo:hi], y[lo:hi], workspace=ws)
    torch.cuda.synchronize()
    close(y, y_r, err)
    close(h, fin, fin_err)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_views_leave_the_rest_alone(cuda, dtype):
    """x | a | b in one wide buffer, outputs in wider ones: neighbours keep their values."""
    lengths, C = [70, 200, 3], 136
    T = sum(lengths)
    inp = make(lengths, C, dtype, seed=8)
    want = gpu_pass(cuda, inp, lengths)
    wide = torch.full((T + 2, 3 * C + 16), float("nan"), dtype=DT[dtype], device=cuda)
    x, ab = wide[1:T + 1, 8:C + 8], wide[1:T + 1, C + 8:3 * C + 8]
    x.copy_(inp["x"]), ab.copy_(inp["ab"])
    out = torch.full((T + 2, 5 * C + 32), 5.0, dtype=DT[dtype], device=cuda)
    y, dx, dab = (out[1:T + 1, i:i + n] for i, n in ((8, C), (C + 16, C), (2 * C + 24, 2 * C)))
    h = inp["h"].clone().to(cuda)
    cu = cu_of(lengths, cuda)
    ws = workspace(la.gated_scan_workspace_bytes, 3, T, C, DT[dtype], dev=cuda)
    saved = workspace(la.gated_scan_saved_bytes, 3, T, C, DT[dtype], dev=cuda)
    dfin, dh0 = inp["dfinal"].to(cuda), torch.empty(3, C, device=cuda)
    la.gated_scan(la.pointer_array(list(h)), x, ab, y, cu, saved=saved, workspace=ws)
    la.gated_scan_backward(x, ab, saved, inp["dy"].to(cuda), dx, dab, cu, dh_final_ptrs=la.pointer_array(list(dfin)),
                           dh0_ptrs=la.pointer_array(list(dh0)), workspace=ws)
    torch.cuda.synchronize()
    for got, ref in zip((y, h, dx, dab, dh0), want):
        assert torch.equal(got, ref)
    out[1:T + 1, 8:C + 8] = out[1:T + 1, C + 16:2 * C + 16] = out[1:T + 1, 2 * C + 24:4 * C + 24] = 5.0
    assert torch.all(out == 5.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_that_are_infinite(cuda, dtype):
    """a = -inf, b = -inf: the state passes a token unchanged; a = inf: it is dropped; b = inf: x enters whole."""
    inf = float("inf")
    T, C = 200, 16
    x = torch.randn(T, C, generator=torch.Generator().manual_seed(9)).to(DT[dtype])
    ab = torch.full((T, 2 * C), -inf)
    ab[70, :C], ab[70, C:] = inf, inf  # h_70 = x_70
    ab[150, C:] = inf  # h_150 = h_149 + x_150
    x[20] = 3e38
    h = torch.randn(1, C, generator=torch.Generator().manual_seed(10)).to(cuda)
    h0 = h.clone()
    xd, abd = x.to(cuda), ab.to(DT[dtype]).to(cuda)
    y = torch.empty_like(xd)
    la.gated_scan(la.pointer_array(list(h)), xd, abd, y,
                  workspace=workspace(la.gated_scan_workspace_bytes, 1, T, C, xd.dtype, dev=cuda))
    torch.cuda.synchronize()
    assert torch.equal(y[:70], h0.to(DT[dtype]).expand(70, C))
    assert torch.equal(y[70:150], xd[70].expand(80, C))
    last = xd[70].float() + xd[150].float()
    assert torch.equal(y[150:], last.to(DT[dtype]).expand(50, C)) and torch.equal(h[0], last)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
def test_a_bad_stream_stays_by_itself(cuda, dtype, poison):
    """NaN or infinities in one stream (inputs, state, gradients) do not reach its neighbours, wherever
    in a tile the streams meet."""
    lengths, C = [10, 30, 200, 20, 0, 64, 300, 100, 5], 24
    inp = make(lengths, C, dtype, seed=11)
    clean = gpu_pass(cuda, inp, lengths)
    ends = np.cumsum([0] + lengths)
    bad = {1, 3, 6}
    for s in bad:
        for n in ("x", "dy"):
            inp[n][ends[s]:ends[s + 1]] = poison
        inp["h"][s] = inp["dfinal"][s] = poison
    got = gpu_pass(cuda, inp, lengths)
    for s in range(len(lengths)):
        if s not in bad:
            rows = slice(ends[s], ends[s + 1])
            for i in (0, 2, 3):
                assert torch.equal(got[i][rows], clean[i][rows]), (s, i)
            for i in (1, 4):
                assert torch.equal(got[i][s], clean[i][s]), (s, i)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_inputs_same_bits_and_streams_independent(cuda, dtype):
    """Repeats agree bit for bit (nothing depends on which block came first)."""
    lengths = [40000, 3, 20000]
    inp = make(lengths, 256, dtype, seed=12, slow=9.0)
    first = gpu_pass(cuda, inp, lengths)
    for _ in range(3):
        for u, v in zip(first, gpu_pass(cuda, inp, lengths)):
            assert torch.equal(u, v)


def test_bad_offsets_stop_the_call(cuda):
    lengths, C = [50, 60, 70], 16
    T = sum(lengths)
    inp = make(lengths, C, "f32", seed=13)
    x, ab, dy = (inp[n].to(cuda) for n in ("x", "ab", "dy"))
    ws = workspace(la.gated_scan_workspace_bytes, 3, T, C, x.dtype, dev=cuda)
    saved = workspace(la.gated_scan_saved_bytes, 3, T, C, x.dtype, dev=cuda)
    for offsets in ([0, 50, 40, T], [1, 50, 110, T], [0, 50, 110, T - 1], [0, 50, T + 5, T], [0, -3, 110, T],
                    [0, 50, 110, 1 << 30]):
        cu = torch.tensor(offsets, dtype=torch.int32, device=cuda)
        h, y, dx, dab = inp["h"].clone().to(cuda), *(torch.full_like(v, 7.0) for v in (x, x, ab))
        la.gated_scan(la.pointer_array(list(h)), x, ab, y, cu, saved=saved, workspace=ws)
        assert la.device_status() == la.LA_DEV_BAD_SEQLENS
        la.gated_scan_backward(x, ab, saved, dy, dx, dab, cu, workspace=ws)
        assert la.device_status() == la.LA_DEV_BAD_SEQLENS
        assert torch.equal(h.cpu(), inp["h"]) and all(bool((v == 7.0).all()) for v in (y, dx, dab))
    assert torch.all(saved == 0xA5)
    got = gpu_pass(cuda, inp, lengths)  # and the next call runs
    close(got[0], *(forward(f64(inp["x"]), f64(inp["ab"])[:, :C], f64(inp["ab"])[:, C:], f64(inp["h"]), lengths)[i] for i in (0, 3)))


def test_graph_replays_and_side_stream(cuda):
    """Captured on a stream of its own with new inputs at every replay; the workspace is shared by two
    graphs that run one after the other."""
    lengths, C = [300, 0, 500, 9], 128
    B, T = len(lengths), sum(lengths)
    cu = cu_of(lengths, cuda)
    ws = workspace(la.gated_scan_workspace_bytes, B, T, C, torch.bfloat16, dev=cuda)
    inps = [make(lengths, C, "bf16", seed=20 + i) for i in range(3)]
    buf = {n: v.to(cuda) for n, v in inps[0].items()}
    saved = workspace(la.gated_scan_saved_bytes, B, T, C, torch.bfloat16, dev=cuda)
    y, dx, dab = (torch.empty_like(buf[n]) for n in ("x", "x", "ab"))
    dh0 = torch.empty_like(buf["dfinal"])
    hp, fp, op = (la.pointer_array(list(v)) for v in (buf["h"], buf["dfinal"], dh0))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(st):
        for k in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                if k == 0:
                    la.gated_scan(hp, buf["x"], buf["ab"], y, cu, saved=saved, workspace=ws)
                else:
                    la.gated_scan_backward(buf["x"], buf["ab"], saved, buf["dy"], dx, dab, cu, dh_final_ptrs=fp,
                                           dh0_ptrs=op, workspace=ws)
            graphs.append(g)
        for inp in inps[1:] + inps:
            for n, v in inp.items():
                buf[n].copy_(v)
            for g in graphs:
                g.replay()
            st.synchronize()
            for u, v in zip((y, buf["h"], dx, dab, dh0), gpu_pass(cuda, inp, lengths)):
                assert torch.equal(u, v)
    assert la.device_status() == 0


def test_two_calls_side_by_side(cuda):
    """Two calls on two streams, each with its own workspace."""
    lengths, C = [20000, 500], 512
    T = sum(lengths)
    inp = make(lengths, C, "bf16", seed=14)
    want = gpu_pass(cuda, inp, lengths)
    x, ab = inp["x"].to(cuda), inp["ab"].to(cuda)
    cu = cu_of(lengths, cuda)
    sides = []
    for _ in range(2):
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        sides.append((st, inp["h"].clone().to(cuda), torch.empty_like(x),
                      workspace(la.gated_scan_workspace_bytes, 2, T, C, x.dtype, dev=cuda)))
    torch.cuda.synchronize()
    ptrs = [la.pointer_array(list(s[1])) for s in sides]
    torch.cuda.synchronize()
    for _ in range(5):
        for (st, h, y, ws), p in zip(sides, ptrs):
            with torch.cuda.stream(st):
                h.copy_(inp["h"], non_blocking=True)
                la.gated_scan(p, x, ab, y, cu, workspace=ws)
    torch.cuda.synchronize()
    for _, h, y, _ in sides:
        assert torch.equal(y, want[0]) and torch.equal(h, want[1])
    assert la.device_status() == 0


def test_offsets_past_32_bits(cuda):
    """Rows whose element offsets pass 2^31 (a row stride of 2^21 elements): the last rows are right."""
    T, C = 1100, 8
    inp = make([T], C, "bf16", seed=15)
    y_r, before, fin, err, err_b, _ = forward(f64(inp["x"]), f64(inp["ab"])[:, :C], f64(inp["ab"])[:, C:], np.zeros((1, C)), [T])
    wide = torch.empty(T, 1 << 21, dtype=torch.bfloat16, device=cuda)
    x, ab, y = wide[:, :C], wide[:, 1024:1024 + 2 * C], wide[:, 4096:4096 + C]
    x.copy_(inp["x"]), ab.copy_(inp["ab"])
    ws = workspace(la.gated_scan_workspace_bytes, 1, T, C, x.dtype, dev=cuda)
    saved = workspace(la.gated_scan_saved_bytes, 1, T, C, x.dtype, dev=cuda)
    la.gated_scan(None, x, ab, y, saved=saved, workspace=ws)
    torch.cuda.synchronize()
    close(y, y_r, err, "bf16")
    dy, dx, dab = wide[:, 8192:8192 + C], wide[:, 9216:9216 + C], wide[:, 10240:10240 + 2 * C]
    dy.copy_(inp["dy"])
    la.gated_scan_backward(x, ab, saved, dy, dx, dab, workspace=ws)
    torch.cuda.synchronize()
    dx_r, dab_r, _ = backward(f64(inp["x"]), f64(inp["ab"])[:, :C], f64(inp["ab"])[:, C:], before, err_b, f64(inp["dy"]), np.zeros((1, C)), [T])
    close(dx, *dx_r, "bf16")
    close(dab, *dab_r, "bf16")


# ------------------------------------------------------------------------------------ decode step
def conv_rows(window, x, w, bias):
    """SiLU of the causal convolution of one token per stream, and the bound of its error: K products
    and sums, then SiLU's sigmoid (argument rounded: |p| 2^-24) and two roundings."""
    xh = np.concatenate([window, x[:, None]], 1)
    p = bias + np.einsum("bkc,ck->bc", xh, w)
    size = abs(bias) + np.einsum("bkc,ck->bc", abs(xh), abs(w))
    out = p * sigmoid(p)
    return out, 2.0 ** -21 * size * 1.2 + (2.0 ** -21 + abs(p) * 2.0 ** -23) * abs(out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("B,C", [(1, 8), (3, 264), (130, 72)])
def test_step(cuda, B, C, K, dtype):
    inp = make([B], C, dtype, seed=30 + K)  # B tokens, one per stream
    g = torch.Generator().manual_seed(31)
    h = torch.randn(B, C, generator=g)
    window = torch.randn(B, max(K - 1, 0), C, generator=g).to(DT[dtype])
    w = (0.5 * torch.randn(C, max(K, 1), generator=g)).to(DT[dtype])
    bias = torch.randn(C, generator=g).to(DT[dtype]) if K != 2 else None
    x, ab = f64(inp["x"]), f64(inp["ab"])
    u, u_err = conv_rows(f64(window), x, f64(w), f64(bias) if bias is not None else 0.0) if K else (x, 0.0)
    d, beta = sigmoid(ab[:, :C]), sigmoid(ab[:, C:])
    want = (1 - d) * f64(h) + beta * u
    err = EPS * (d * abs(f64(h)) + beta * abs(u)) + UPDATE * (abs(f64(h)) + beta * abs(u)) + beta * u_err
    hd, wd = h.clone().to(cuda), window.clone().to(cuda)
    # rows of a wider buffer
    xd = torch.zeros(B, C + 8, dtype=DT[dtype], device=cuda)[:, :C].copy_(inp["x"])
    y = torch.full((B, C + 16), 5.0, dtype=DT[dtype], device=cuda)
    la.gated_scan_step(la.pointer_array(list(hd)), xd, inp["ab"].to(cuda), y[:, 8:C + 8],
                       conv_state_ptrs=la.pointer_array(list(wd)) if K > 1 else None,
                       conv_w=w.to(cuda) if K else None, conv_bias=bias.to(cuda) if K and bias is not None else None)
    torch.cuda.synchronize()
    close(hd, want, err)
    close(y[:, 8:C + 8], want, err, dtype)
    assert torch.all(y[:, :8] == 5.0) and torch.all(y[:, C + 8:] == 5.0)
    if K > 1:
        assert torch.equal(wd.cpu(), torch.cat([window[:, 1:], inp["x"][:, None]], 1))


def test_steps_follow_a_prefill(cuda):
    """A prompt through the scan, then tokens one by one: y and the state are the whole sequence's."""
    T, n, C = 300, 5, 72
    inp = make([T + n], C, "f32", seed=33, slow=6.0)
    y_r, _, fin, err, _, fin_err = forward(f64(inp["x"]), f64(inp["ab"])[:, :C], f64(inp["ab"])[:, C:], f64(inp["h"]), [T + n])
    x, ab, h = (inp[k].clone().to(cuda) for k in ("x", "ab", "h"))
    y, p = torch.empty_like(x), la.pointer_array(list(h))
    la.gated_scan(p, x[:T], ab[:T], y[:T], workspace=workspace(la.gated_scan_workspace_bytes, 1, T, C, x.dtype, dev=cuda))
    for t in range(T, T + n):
        la.gated_scan_step(p, x[t:t + 1], ab[t:t + 1], y[t:t + 1])
    torch.cuda.synchronize()
    close(y, y_r, err)
    close(h, fin, fin_err)
