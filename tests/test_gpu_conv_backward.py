"""The backward pass of the causal conv1d + SiLU on the GPU against a plain form in 64 bits.

Bounds: p is a sum of K + 1 terms in 32 bits, off by at most 5 * 2^-24 of the sum of their magnitudes P;
SiLU' changes by at most 0.5 of that (its slope is under 0.5), and its own evaluation (sigmoid with
the rounded argument |p| 2^-24, hardware exponential and reciprocal 2^-22 + 2^-23, a few roundings)
stays under (2^-20 + |p| 2^-22). A sum of n terms adds n 2^-24 of their magnitudes at most.
"""
import numpy as np
import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la
from tests.helpers import f64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def reference(window, x, w, bias, dout, dfinal, lengths):
    """Values and error bounds of dx, dw, dbias and the windows' gradients."""
    C, K = w.shape
    dx, dx_e = np.zeros_like(x), np.zeros_like(x)
    dw, dw_e, db, db_e = np.zeros((C, K)), np.zeros((C, K)), np.zeros(C), np.zeros(C)
    dwin, dwin_e = np.zeros_like(window), np.zeros_like(window)
    t0 = 0
    for s, n in enumerate(lengths):
        xh = np.concatenate([window[s], x[t0:t0 + n]])
        g, g_e = np.zeros_like(xh), np.zeros_like(xh)
        for t in range(n):
            rows = xh[t:t + K]
            p = bias + (rows * w.T).sum(0)
            size = abs(bias) + abs(rows * w.T).sum(0)
            sg = 1 / (1 + np.exp(-p))
            dp = dout[t0 + t] * sg * (1 + p * (1 - sg))
            e = abs(dout[t0 + t]) * (2.0 ** -20 + abs(p) * 2.0 ** -22 + 5 * 2.0 ** -24 * size)
            g[t:t + K] += dp * w.T
            g_e[t:t + K] += (e + K * 2.0 ** -24 * abs(dp)) * abs(w.T)
            dw += (dp * rows).T
            dw_e += ((e + 2.0 ** -22 * abs(dp)) * abs(rows)).T
            db += dp
            db_e += e + 2.0 ** -22 * abs(dp)
        if K > 1:
            g[n:] += dfinal[s]
            g_e[n:] += K * 2.0 ** -24 * abs(dfinal[s])
        dwin[s], dwin_e[s] = g[:K - 1], g_e[:K - 1]
        dx[t0:t0 + n], dx_e[t0:t0 + n] = g[K - 1:], g_e[K - 1:]
        t0 += n
    # the sums over tokens: runs of at most 256, then the runs, each under 2^-24 of the magnitudes a term
    # in the worst case; 2^-22 a term above is already counted, long sums of one sign add the square root
    return (dx, dx_e), (dw, dw_e), (db, db_e), (dwin, dwin_e)


def close(got, want, err, dtype="f32"):
    got = f64(got)
    assert np.all(np.isfinite(got))
    tol = err + HALF[dtype] * (abs(want) + err) + 1e-37
    worst = np.max(abs(got - want) / tol) if got.size else 0.0
    assert worst <= 1, worst


def make(lengths, C, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    T, B = sum(lengths), len(lengths)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(window=r(B, K - 1, C).to(DT[dtype]), x=r(T, C).to(DT[dtype]), w=(0.5 * r(C, K)).to(DT[dtype]),
                bias=r(C).to(DT[dtype]), dout=r(T, C).to(DT[dtype]), dfinal=r(B, K - 1, C).to(DT[dtype]))


def gpu_pass(cuda, inp, lengths, *, packed=True, bias=True, states=True):
    T, C = inp["x"].shape
    K, B, dt = inp["w"].shape[1], len(lengths), inp["x"].dtype
    d = {n: v.to(cuda) for n, v in inp.items()}
    dx = torch.full_like(d["x"], 7.0)
    dw, db = torch.full((C, K), 7.0, device=cuda), torch.full((C,), 7.0, device=cuda)
    dwin = torch.full_like(d["window"], 7.0)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=cuda) if packed else None
    ws = torch.empty(la.conv1d_silu_backward_workspace_bytes(B, T, C, K, dt), dtype=torch.uint8, device=cuda).fill_(0xFF)
    p = lambda v: la.pointer_array(list(v)) if K > 1 else None  # noqa: E731
    la.conv1d_silu_backward(p(d["window"]), d["x"], d["w"], d["dout"], dx, dw, cu, B=B,
                            bias=d["bias"] if bias else None, dbias=db if bias else None,
                            dstate_final_ptrs=p(d["dfinal"]) if states else None,
                            dstate_ptrs=p(dwin) if states else None, workspace=ws)
    torch.cuda.synchronize()
    assert la.device_status() == 0
    return dx, dw, db, dwin


LENGTHS = {"one": [1], "two": [2], "three": [3], "run": [64], "run+1": [65], "batch": [130, 130], "ones": [1] * 9,
           "ragged": [0, 1, 2, 0, 3, 4, 63, 64, 65, 0, 257, 0], "long": [1500]}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("name", LENGTHS)
def test_conv_backward(cuda, name, K, dtype):
    lengths, C = LENGTHS[name], {1: 8, 2: 72, 3: 520, 4: 136}[K]
    inp = make(lengths, C, K, dtype, seed=K + len(name))
    ref = reference(*(f64(inp[n]) for n in ("window", "x", "w", "bias", "dout", "dfinal")), lengths)
    dx, dw, db, dwin = gpu_pass(cuda, inp, lengths, packed=name != "batch")
    close(dx, *ref[0], dtype)
    close(dw, *ref[1])
    close(db, *ref[2])
    close(dwin, *ref[3], dtype)


def test_without_bias_and_states(cuda):
    lengths = [5, 0, 200, 2]
    inp = make(lengths, 40, 4, "f32", seed=3)
    v = {n: f64(inp[n]) for n in inp}
    ref = reference(v["window"], v["x"], v["w"], 0 * v["bias"], v["dout"], 0 * v["dfinal"], lengths)
    dx, dw, db, dwin = gpu_pass(cuda, inp, lengths, bias=False, states=False)
    close(dx, *ref[0])
    close(dw, *ref[1])
    assert torch.all(db == 7.0) and torch.all(dwin == 7.0)


def test_gradients_against_differences_of_the_forward_kernel(cuda):
    """Differences of the library's own forward pass in fp32, of a loss over its outputs and the
    windows it leaves. With a step of 1/32 the third derivative (SiLU''' under 0.6, |w| under 2) leaves
    0.6 * 8 / 6 / 1024 of |dout| for each of K outputs; rounding 2^-21 * 10 * 32."""
    lengths, C, K = [3, 0, 6], 8, 4
    inp = make(lengths, C, K, "f32", seed=4)
    inp["w"].clamp_(-1, 1)
    cu = torch.tensor([0, 3, 3, 9], dtype=torch.int32, device=cuda)

    def loss(v):
        st = v["window"].clone().to(cuda)
        out = torch.empty(9, C, device=cuda)
        la.conv1d_silu_prefill_varlen(la.pointer_array(list(st)), v["x"].to(cuda), v["w"].to(cuda), out, cu,
                                      bias=v["bias"].to(cuda))
        return float((f64(out) * f64(inp["dout"])).sum() + (f64(st) * f64(inp["dfinal"])).sum())

    dx, dw, db, dwin = gpu_pass(cuda, inp, lengths)
    step = 1.0 / 32
    rng = np.random.default_rng(4)
    for name, got in (("x", dx), ("w", dw), ("bias", db), ("window", dwin)):
        got = f64(got)
        places = list(np.ndindex(got.shape))
        for i in (places[j] for j in rng.choice(len(places), min(12, len(places)), replace=False)):
            up, down = ({k: u.clone() for k, u in inp.items()} for _ in range(2))
            up[name][i] += step
            down[name][i] -= step
            want = (loss(up) - loss(down)) / (2 * step)
            n_out = 9 if name in ("w", "bias") else K
            size = 3.0 ** 3 if name == "w" else 1.0  # the rows that multiply a tap: |x| under 3.5
            assert abs(got[i] - want) <= n_out * 3.5 * size * (0.6 / 6 * step ** 2) + 1e-3, (name, i, got[i], want)


def test_repeats_strides_and_neighbours(cuda):
    lengths, C, K = [700, 1, 0, 900], 136, 4
    T = sum(lengths)
    inp = make(lengths, C, K, "bf16", seed=5)
    want = gpu_pass(cuda, inp, lengths)
    for u, v in zip(want, gpu_pass(cuda, inp, lengths)):
        assert torch.equal(u, v)
    wide = torch.full((T + 2, 3 * C + 24), 5.0, dtype=torch.bfloat16, device=cuda)
    x, dout, dx = (wide[1:T + 1, i:i + C] for i in (8, C + 8, 2 * C + 16))
    x.copy_(inp["x"]), dout.copy_(inp["dout"])
    before = wide.clone()
    win, fin = inp["window"].to(cuda), inp["dfinal"].to(cuda)
    dwin, dw, db = torch.empty_like(win), torch.empty(C, K, device=cuda), torch.empty(C, device=cuda)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=cuda)
    ws = torch.empty(la.conv1d_silu_backward_workspace_bytes(4, T, C, K, x.dtype), dtype=torch.uint8, device=cuda)
    la.conv1d_silu_backward(la.pointer_array(list(win)), x, inp["w"].to(cuda), dout, dx, dw, cu,
                            bias=inp["bias"].to(cuda), dbias=db, dstate_final_ptrs=la.pointer_array(list(fin)),
                            dstate_ptrs=la.pointer_array(list(dwin)), workspace=ws)
    torch.cuda.synchronize()
    for u, v in zip((dx, dw, db, dwin), want):
        assert torch.equal(u, v)
    assert torch.equal(win.cpu(), inp["window"]) and torch.equal(fin.cpu(), inp["dfinal"])
    dx.copy_(before[1:T + 1, 2 * C + 16:3 * C + 16])
    assert torch.equal(wide, before)


def test_a_bad_stream_stays_by_itself(cuda):
    """NaN in one stream: the others' dx and windows are as they were (dw and dbias sum over all)."""
    lengths, C, K = [100, 3, 70, 1, 64], 24, 4
    inp = make(lengths, C, K, "bf16", seed=6)
    clean = gpu_pass(cuda, inp, lengths)
    ends = np.cumsum([0] + lengths)
    for s in (1, 3):
        for n in ("x", "dout"):
            inp[n][ends[s]:ends[s + 1]] = float("nan")
        inp["window"][s] = inp["dfinal"][s] = float("nan")
    got = gpu_pass(cuda, inp, lengths)
    for s in (0, 2, 4):
        assert torch.equal(got[0][ends[s]:ends[s + 1]], clean[0][ends[s]:ends[s + 1]])
        assert torch.equal(got[3][s], clean[3][s])


def test_far_values_stay_finite(cuda):
    """|p| beyond the exponential's range: SiLU' is 1 or 0, not NaN."""
    C = 8
    x = torch.full((4, C), 200.0)
    x[2:] = -200.0
    inp = dict(window=torch.zeros(1, 0, C), x=x, w=torch.ones(C, 1), bias=torch.zeros(C), dout=torch.ones(4, C),
               dfinal=torch.zeros(1, 0, C))
    dx, dw, db, _ = gpu_pass(cuda, inp, [4])
    assert torch.equal(dx.cpu(), torch.tensor([1.0, 1.0, 0.0, 0.0])[:, None].expand(4, C))
    assert torch.equal(dw.cpu(), torch.full((C, 1), 400.0)) and torch.equal(db.cpu(), torch.full((C,), 2.0))


def test_bad_offsets_stop_the_call(cuda):
    inp = {n: v.to(cuda) for n, v in make([40, 60], 16, 4, "f32", seed=7).items()}
    for offsets in ([0, 70, 60], [1, 40, 100], [0, 40, 99], [0, -1, 100], [0, 101, 100]):
        cu = torch.tensor(offsets, dtype=torch.int32, device=cuda)
        dx, dw, db = torch.full_like(inp["x"], 7.0), torch.full((16, 4), 7.0, device=cuda), torch.full((16,), 7.0, device=cuda)
        dwin = torch.full_like(inp["window"], 7.0)
        ws = torch.empty(la.conv1d_silu_backward_workspace_bytes(2, 100, 16, 4, dx.dtype), dtype=torch.uint8, device=cuda)
        la.conv1d_silu_backward(la.pointer_array(list(inp["window"])), inp["x"], inp["w"], inp["dout"], dx, dw, cu,
                                dbias=db, dstate_ptrs=la.pointer_array(list(dwin)), workspace=ws)
        assert la.device_status() == la.LA_DEV_BAD_SEQLENS
        assert all(bool((v == 7.0).all()) for v in (dx, dw, db, dwin))


def test_graph_replay(cuda):
    lengths, C, K = [100, 0, 300], 64, 4
    inps = [make(lengths, C, K, "bf16", seed=40 + i) for i in range(2)]
    buf = {n: v.to(cuda) for n, v in inps[0].items()}
    dx, dw, db, dwin = torch.empty_like(buf["x"]), torch.empty(C, K, device=cuda), torch.empty(C, device=cuda), torch.empty_like(buf["window"])
    ptrs = [la.pointer_array(list(v)) for v in (buf["window"], buf["dfinal"], dwin)]
    cu = torch.tensor([0, 100, 100, 400], dtype=torch.int32, device=cuda)
    ws = torch.empty(la.conv1d_silu_backward_workspace_bytes(3, 400, C, K, dx.dtype), dtype=torch.uint8, device=cuda)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        la.conv1d_silu_backward(ptrs[0], buf["x"], buf["w"], buf["dout"], dx, dw, cu, bias=buf["bias"], dbias=db,
                                dstate_final_ptrs=ptrs[1], dstate_ptrs=ptrs[2], workspace=ws)
    for inp in inps[::-1] + inps:
        for n, v in inp.items():
            buf[n].copy_(v)
        g.replay()
        torch.cuda.synchronize()
        for u, v in zip((dx, dw, db, dwin), gpu_pass(cuda, inp, lengths)):
            assert torch.equal(u, v)


@pytest.mark.parametrize("B", [1003, 990, 979])
def test_long_runs_of_tokens_and_many_empty_streams(cuda, B):
    """The runs' length follows the call's sizes: 384 tokens with 1003 streams, 192 with 990, 96 with 979.
    Streams that end just before, at and after such a run's end, among empty ones."""
    lengths = [0] * B
    for at, n in ((0, 95), (3, 96), (4, 97), (200, 191), (201, 193), (500, 383), (777, 385), (B - 1, 770)):
        lengths[at] = n
    assert sum(lengths) == 2210
    inp = make(lengths, 8, 4, "f32", seed=B)
    ref = reference(*(f64(inp[n]) for n in ("window", "x", "w", "bias", "dout", "dfinal")), lengths)
    for got, want in zip(gpu_pass(cuda, inp, lengths), ref):
        close(got, *want)
