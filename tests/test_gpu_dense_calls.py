"""The dense half's calls as programs make them: many tiles, long sums, far strides, shared buffers, other streams,
captured graphs, values that are not finite, bounded waits, and the whole block (FeedForward) against 64 bits and
against differences of its 64-bit form. Bounds are those of test_gpu_dense.py, or stated where they are used."""
import math

import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la
from linear_attention_chunked_conv1d_gb300.path import FeedForward
from tests.test_gpu_dense import F32, U, act64, case, check_gated, check_linear, close, gated_case, out_rows, room, rows

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


# tiles of 256 x 256 that go round the pairs more than once, with ragged edges; and sums that are split over blocks
@pytest.mark.parametrize("m,n,k", [(1030, 4100, 136), (2500, 2600, 264), (4099, 2733, 65), (9000, 600, 520), (5000, 300, 2100), (130, 130, 8200)])
def test_linear_many_tiles(cuda, m, n, k):
    check_linear(case(cuda, m, n, k, m + n + k), "none")
    check_linear(case(cuda, m, n, k, m + n + k + 1, residual=False), "gelu")


@pytest.mark.parametrize("m,f,k", [(1030, 2100, 136), (2500, 1300, 264), (4099, 2733, 65), (9000, 300, 520), (5000, 150, 2100), (130, 130, 8200)])
def test_gated_many_tiles(cuda, m, f, k):
    check_gated(gated_case(cuda, m, f, k, m + f + k), "silu")


@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129])
def test_rows_around_the_tiles(cuda, m):
    check_linear(case(cuda, m, 392, 1100, m), "silu")
    check_gated(gated_case(cuda, m, 197, 1100, m), "gelu_tanh")


@pytest.mark.parametrize("m,n,k", [(777, 5001, 2048), (1030, 8192, 2048), (777, 2048, 5001), (257, 2000, 520), (1281, 3000, 136), (513, 392, 2100), (4099, 4500, 72)])
def test_a_few_rows_past_whole_tiles(cuda, m, n, k):
    """The rows past the last whole tile may be another kernel's, beside the first one's last round: between calls that
    write what it reads and read what it writes, with nothing of the one's rows missing or touched by the other."""
    c = case(cuda, m, n, k, m)
    check_linear(c, "gelu")
    check_linear(case(cuda, m, n, k, m + 1, bias=False, residual=False), "none")
    g = gated_case(cuda, m, n, k, m + 2)
    check_gated(g, "silu")
    want = c["dx"].double()  # of the call that makes dw too
    c["dx"].fill_(7.0)
    saved = room(la.linear_saved_bytes(m, n, "gelu"), cuda)
    la.linear(c["x"], c["w"], bias=c["bias"], act="gelu", saved=saved)
    la.linear_backward(c["x"], c["w"], saved, c["dy"], c["dx"], act="gelu", workspace=room(la.linear_backward_workspace_bytes(m, n, k, "gelu"), cuda))
    assert float((c["dx"].double() - want).norm()) <= 2 * U * float(want.norm())  # one rounding each
    # in the residual's place
    res = rows_like(c["residual"])
    assert torch.equal(la.linear(c["x"], c["w"], res, bias=c["bias"], residual=res, act="gelu"), la.linear(c["x"], c["w"], bias=c["bias"], residual=c["residual"], act="gelu"))
    # a chain on one stream, eager and replayed: x is written by the call before, y read by the next and written again
    w2 = (torch.randn(k, n, device=cuda) / math.sqrt(n)).to(BF16)
    if n % 8 or k % 8:
        w2 = rows_like(w2)
    x0, x1, y, z = rows_like(c["x"]), rows_like(c["x"]), out_rows((m, n), BF16, cuda), out_rows((m, k), BF16, cuda)

    def chain():
        x1.copy_(x0)
        for _ in range(3):
            la.linear(x1, c["w"], y, bias=c["bias"], act="silu")
            la.linear(y, w2, z)
            la.layernorm_rows(z, torch.ones(k, dtype=BF16, device=cuda), y=x1)
        return x1.clone()
    cur = x0
    for _ in range(3):
        a = la.linear(cur, c["w"], bias=c["bias"], act="silu")
        torch.cuda.synchronize()
        b = la.linear(a, w2)
        torch.cuda.synchronize()
        cur = la.layernorm_rows(b, torch.ones(k, dtype=BF16, device=cuda))
        torch.cuda.synchronize()
    for _ in range(5):
        assert torch.equal(chain(), cur)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for _ in range(5):
        out.zero_()
        graph.replay()
        assert torch.equal(out, cur)
    # two chains at once, on streams of their own
    u, v = torch.cuda.Stream(), torch.cuda.Stream()
    ends = [torch.empty(m, (k + 7) // 8 * 8, dtype=BF16, device=cuda)[:, :k] for _ in range(2)]
    mids = [out_rows((m, n), BF16, cuda) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(6):
        for st, mid, end in zip((u, v), mids, ends):
            la.linear(x0, c["w"], mid, bias=c["bias"], act="silu", stream=st)
            la.linear(mid, w2, end, stream=st)
    torch.cuda.synchronize()
    first = la.linear(la.linear(x0, c["w"], bias=c["bias"], act="silu"), w2)
    assert all(torch.equal(end, first) for end in ends)
    assert la.device_status() == 0


@pytest.mark.parametrize("m,n,k", [(16384, 520, 392), (30001, 257, 264), (8192, 256, 256), (12000, 1001, 513), (40000, 8, 72)])
def test_long_sums_of_small_weights(cuda, m, n, k):
    """dw's sum over many rows in parts that are joined, next to dx and alone, the same bits each time; the workspace
    starts as NaN and what the parts do not reach is not read."""
    c = case(cuda, m, n, k, m)
    check_linear(c, "gelu")
    check_gated(gated_case(cuda, m, n, k, m + 1), "silu")
    nan = lambda b: torch.full((b // 4 + 4,), float("nan"), device=cuda).view(torch.uint8)  # noqa: E731
    ref = c["dy"].double().T @ c["x"].double()
    mag = c["dy"].double().abs().T @ c["x"].double().abs()
    got = []
    for dx in (None, c["dx"], None):
        c["dw"].fill_(7.0)
        la.linear_backward(c["x"], c["w"], None, c["dy"], dx, c["dw"], workspace=nan(la.linear_backward_workspace_bytes(m, n, k)))
        # sums of m terms in parts of at least 512, each in fp32: (m / 8) 2^-24 of the terms is far more than their order adds
        close(c["dw"], ref, U * ref.abs() + max(64, m / 8) * F32 * mag, "dw")
        got.append(c["dw"].clone())
    assert torch.equal(got[0], got[2])
    assert la.device_status() == 0


def test_far_strides(cuda):
    """Rows 2^31 values apart: offsets pass 32 bits in x, residual and y, in dy and dx, and in a norm's rows."""
    g = torch.Generator().manual_seed(1)
    far = 2 ** 31
    big = torch.empty(2 * far + 4096, dtype=BF16, device=cuda)
    at = lambda o, r, c: big.as_strided((r, c), (far, 1), o)  # noqa: E731
    m, n, k = 3, 72, 200
    x, y, res, dy, dx = at(0, m, k), at(256, m, n), at(512, m, n), at(768, m, n), at(1024, m, k)
    for t in (x, res, dy):
        t.copy_(torch.randn(t.shape, generator=g).to(BF16))
    w = (torch.randn(n, k, generator=g) / math.sqrt(k)).to(BF16).to(cuda)
    dw = torch.empty_like(w)
    want_y = la.linear(x.contiguous(), w, residual=res.contiguous())
    want_dx, want_dw = torch.empty(m, k, dtype=BF16, device=cuda), torch.empty_like(w)
    ws = room(la.linear_backward_workspace_bytes(m, n, k), cuda)
    la.linear_backward(x.contiguous(), w, None, dy.contiguous(), want_dx, want_dw, workspace=ws)
    assert torch.equal(la.linear(x, w, y, residual=res), want_y)
    la.linear_backward(x, w, None, dy, dx, dw, workspace=ws)
    assert torch.equal(dx, want_dx) and torch.equal(dw, want_dw)
    nw = torch.ones(k, dtype=BF16, device=cuda)
    assert torch.equal(la.layernorm_rows(x, nw, None, dx), la.layernorm_rows(x.contiguous(), nw))


def test_shared_buffers(cuda):
    """Halves of one packed weight and gradient, operands and results as columns of one buffer, y in the residual's
    place; each as the call with buffers of their own."""
    g = torch.Generator().manual_seed(2)
    m, f, k = 700, 328, 264
    x = rows((m, k), BF16, cuda, g)
    w = rows((2 * f, k), BF16, cuda, g, 1 / math.sqrt(k))
    dh = rows((m, f), BF16, cuda, g)
    saved, ws = room(la.gated_ffn_saved_bytes(m, f), cuda), room(la.gated_ffn_backward_workspace_bytes(m, f, k), cuda)
    h = la.gated_ffn(x, w[:f].clone(), w[f:].clone(), saved=saved)
    dx, dg, du = (torch.empty(*s, dtype=BF16, device=cuda) for s in ((m, k), (f, k), (f, k)))
    la.gated_ffn_backward(x, w[:f].clone(), w[f:].clone(), saved, dh, dx, dg, du, workspace=ws)
    wide = torch.full((m, k + f + k + 16), 3.0, dtype=BF16, device=cuda)
    x2, h2, dx2 = wide[:, :k], wide[:, k:k + f], wide[:, k + f:2 * k + f]
    x2.copy_(x)
    dw2 = torch.empty(2 * f, k, dtype=BF16, device=cuda)
    la.gated_ffn(x2, w[:f], w[f:], h2, saved=saved)
    la.gated_ffn_backward(x2, w[:f], w[f:], saved, dh, dx2, dw2[:f], dw2[f:], workspace=ws)
    assert torch.equal(h2, h) and torch.equal(dx2, dx) and torch.equal(dw2[:f], dg) and torch.equal(dw2[f:], du)
    assert bool((wide[:, 2 * k + f:] == 3.0).all())
    for rows_ in (m, 5):  # tiles by pairs of blocks, and split sums
        xs, wd, res = x[:rows_], w[:f], rows((rows_, f), BF16, cuda, g)
        want = la.linear(xs, wd, residual=res, act="silu")
        assert la.linear(xs, wd, res, residual=res, act="silu") is res and torch.equal(res, want)


@pytest.mark.parametrize("m,n,k,act", [(700, 520, 264, "gelu"), (5, 520, 264, "none"), (70, 40, 1000, "silu"), (3000, 1100, 264, "none")])
def test_gradients_that_are_asked_for(cuda, m, n, k, act):
    """Any of dx, dw and dbias alone, or two of them, as all three together."""
    c = case(cuda, m, n, k, 21)
    saved = room(la.linear_saved_bytes(m, n, act), cuda) if act != "none" else None
    ws = room(la.linear_backward_workspace_bytes(m, n, k, act), cuda)
    la.linear(c["x"], c["w"], bias=c["bias"], act=act, saved=saved)
    la.linear_backward(c["x"], c["w"], saved, c["dy"], c["dx"], c["dw"], dbias=c["dbias"], act=act, workspace=ws)
    want = [c[q].double() for q in ("dx", "dw", "dbias")]
    for which in range(1, 7):
        got = [torch.full_like(c[q], 7.0, memory_format=torch.preserve_format) if which >> i & 1 else None for i, q in enumerate(("dx", "dw", "dbias"))]
        la.linear_backward(c["x"], c["w"], saved, c["dy"], got[0], got[1], dbias=got[2], act=act, workspace=ws)
        for g, w in zip(got, want):
            # one launch or two may split a sum differently: last places of fp32 sums, then one rounding
            assert g is None or float((g.double() - w).norm()) <= 2 * U * float(w.norm())
    f = gated_case(cuda, m, n, k, 22)
    saved, ws = room(la.gated_ffn_saved_bytes(m, n), cuda), room(la.gated_ffn_backward_workspace_bytes(m, n, k), cuda)
    la.gated_ffn(f["x"], f["w"], f["w_up"], saved=saved)
    la.gated_ffn_backward(f["x"], f["w"], f["w_up"], saved, f["dy"], f["dx"], f["dw"], f["dw_up"], workspace=ws)
    want = [f[q].double() for q in ("dx", "dw", "dw_up")]
    for q in ("dx", "dw", "dw_up"):
        f[q].fill_(7.0)
    la.gated_ffn_backward(f["x"], f["w"], f["w_up"], saved, f["dy"], f["dx"], workspace=ws)
    la.gated_ffn_backward(f["x"], f["w"], f["w_up"], saved, f["dy"], None, f["dw"], f["dw_up"], workspace=ws)
    for q, w in zip(("dx", "dw", "dw_up"), want):
        assert float((f[q].double() - w).norm()) <= 2 * U * float(w.norm())


def test_one_row_one_column_and_one_of_each(cuda):
    """A single row goes with any stride, its own width's among them, and so does a weight of one output."""
    g = torch.Generator().manual_seed(23)
    x = torch.randn(1, 77, generator=g).to(BF16).to(cuda)
    w = torch.randn(30, 80, generator=g).to(BF16).to(cuda)[:, :77]
    y = torch.empty(1, 30, dtype=BF16, device=cuda)
    ref = x.double() @ w.double().T
    bound = U * ref.abs() + 64 * F32 * (x.double().abs() @ w.double().abs().T)
    close(la.linear(x, w, y), ref, bound, "y")
    one = torch.randn(1, 77, generator=g).to(BF16).to(cuda)
    out = torch.empty(1, 1, dtype=BF16, device=cuda)
    ref = x.double() @ one.double().T
    close(la.linear(x, one, out), ref, U * ref.abs() + 64 * F32 * (x.double().abs() @ one.double().abs().T), "1 x 1")
    dx, dw = torch.empty_like(x), torch.empty_like(one)
    dy = torch.ones(1, 1, dtype=BF16, device=cuda)
    la.linear_backward(x, one, None, dy, dx, dw, workspace=room(la.linear_backward_workspace_bytes(1, 1, 77), cuda))
    assert torch.equal(dx, one) and torch.equal(dw, x)
    h = la.gated_ffn(x, one, one)
    a = ref * torch.sigmoid(ref) * ref
    close(h, a, U * a.abs() + 1e-4 * a.abs().clamp(min=1e-3), "h")  # 64 2^-24 of sums of 77 terms, three times over: 1e-5 of them
    st = torch.empty(1, 2, device=cuda)
    assert la.layernorm_rows(x, torch.ones(77, dtype=BF16, device=cuda), stats=st).shape == (1, 77)


def test_first_calls_of_a_process_inside_a_capture(cuda):
    """Nothing is set up by a first call that a capture would not allow."""
    import subprocess
    import sys
    code = """
import torch
import linear_attention_chunked_conv1d_gb300 as la
b = torch.bfloat16
x, w, u = (torch.randn(2000, 512, device="cuda").to(b) for _ in range(3))
n, o, s, h, dx = torch.ones(512, device="cuda").to(b), torch.empty_like(x), torch.empty(2000, 2000, device="cuda", dtype=b), torch.empty(2000, 2000, device="cuda", dtype=b), torch.empty_like(x)
few, ws = torch.empty(3, 2000, device="cuda", dtype=b), torch.empty(la.linear_backward_workspace_bytes(2000, 2000, 512), device="cuda", dtype=torch.uint8)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    la.layernorm_rows(x, n, y=o)
    la.linear(o, w, s)
    la.gated_ffn(o, w, u, h)
    la.linear(o[:3], w, few)
    la.linear_backward(o, w, None, h, dx, workspace=ws)
for t in (o, s, h, few, dx):
    t.zero_()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (o, s, h, few, dx)]
la.layernorm_rows(x, n, y=o), la.linear(o, w, s), la.gated_ffn(o, w, u, h), la.linear(o[:3], w, few), la.linear_backward(o, w, None, h, dx, workspace=ws)
assert la.device_status() == 0 and all(torch.equal(p, q) for p, q in zip(got, (o, s, h, few, dx)))
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_same_bits_each_time(cuda):
    """Sums are taken in a fixed order: every call, in whatever company, gives the same bits."""
    c, d = gated_case(cuda, 2000, 700, 520, 3), case(cuda, 40, 500, 2000, 4)
    first = None
    for _ in range(5):
        saved, ws = room(la.gated_ffn_saved_bytes(2000, 700), cuda), room(la.gated_ffn_backward_workspace_bytes(2000, 700, 520), cuda)
        la.gated_ffn(c["x"], c["w"], c["w_up"], c["y"], saved=saved)
        la.gated_ffn_backward(c["x"], c["w"], c["w_up"], saved, c["dy"], c["dx"], c["dw"], c["dw_up"], workspace=ws)
        la.linear(d["x"], d["w"], d["y"], bias=d["bias"], act="gelu")
        stats, dw, db = torch.empty(2000, 2, device=cuda), torch.empty(520, device=cuda), torch.empty(520, device=cuda)
        nw = torch.ones(520, dtype=BF16, device=cuda)
        la.layernorm_rows(c["x"], nw, stats=stats)
        dn = torch.empty(2000, 520, dtype=BF16, device=cuda)
        la.layernorm_rows_backward(c["x"], nw, stats, c["dx"], dn, dw, db,
                                   workspace=room(la.layernorm_rows_backward_workspace_bytes(2000, 520, BF16), cuda))
        got = [t.clone() for t in (c["y"], c["dx"], c["dw"], c["dw_up"], d["y"], dn, dw, db)]
        assert first is None or all(torch.equal(a, b) for a, b in zip(first, got))
        first = first or got


def test_a_row_does_not_depend_on_its_batch_mates(cuda):
    """Rows of NaN and infinities leave the other rows of y and dx as they are; a weight's row of NaN its column."""
    for m in (12, 900):
        c = gated_case(cuda, m, 300, 200, 5)
        run = lambda: la.gated_ffn(c["x"], c["w"], c["w_up"]).clone()  # noqa: E731
        good = run()
        c["x"][3], c["x"][7, 5] = float("nan"), float("inf")
        c["w"][11] = float("nan")
        got = run()
        keep_m, keep_n = [i for i in range(m) if i not in (3, 7)], [i for i in range(300) if i != 11]
        assert torch.equal(got[keep_m][:, keep_n], good[keep_m][:, keep_n])
        assert got[3].isnan().all() and got[:, 11].isnan().all()
        assert not got[7][keep_n].isfinite().any()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_large_and_special_values_of_activations(cuda, act):
    """z from -1e30 to 1e30 through a weight of 1 x 1: values and slopes go to their limits, never to NaN."""
    z = torch.tensor([-1e30, -3e8, -1e4, -300, -90, -60, -20, -9, -5, -1, -0.1, -1e-3, -1e-30, 0.0, 1e-30, 1e-3, 0.1, 1, 5, 9, 20, 300, 1e4, 1e30])
    x = z.to(BF16).reshape(-1, 1).to(cuda).expand(-1, 8).contiguous()[:, :1]
    w = torch.ones(1, 8, dtype=BF16, device=cuda)[:, :1]
    m = z.numel()
    saved, dy, dx = room(la.linear_saved_bytes(m, 1, act), cuda), torch.ones(m, 8, dtype=BF16, device=cuda)[:, :1], torch.zeros(m, 8, dtype=BF16, device=cuda)[:, :1]
    y = la.linear(x, w, act=act, saved=saved)
    la.linear_backward(x, w, saved, dy, dx, act=act, workspace=room(la.linear_backward_workspace_bytes(m, 1, 1, act), cuda))
    X = x.double().clamp(-1e9, 1e9) if act != "relu" else x.double()
    X.requires_grad_()
    ref = act64(X, act)
    slope = torch.autograd.grad(ref.sum(), X)[0]
    ref = torch.where(x.double() > 1e8, x.double(), ref.detach())
    # 2^-17: the hardware's exponential and reciprocal, and an exponent z^2 / 2 rounded to 2^-24 of at most 2^6. The factor
    # of z is a 32-bit number whose values below 2^-126 count as 0 (silu at -90: 90 e^-90 = 90 * 8.2e-40 with e^-90 < 2^-126
    # = 1.2e-38), so what is lost of z times it is at most |z| 2^-126, where that is not past the range of z itself.
    close(y, ref, U * ref.abs() + 2.0 ** -17 * ref.abs() + x.double().abs().clamp(max=200) * 2.0 ** -126 + 1e-38, "value")
    if act == "relu":
        slope = (x.double() > 0).double()
    close(dx, slope, U * slope.abs() + 2.0 ** -20, "slope")


def test_other_streams_and_two_at_once(cuda):
    c, d = gated_case(cuda, 1500, 600, 520, 6), gated_case(cuda, 1500, 600, 520, 7)

    def run(q, stream):
        q["saved"], q["ws"] = room(la.gated_ffn_saved_bytes(1500, 600), cuda), room(la.gated_ffn_backward_workspace_bytes(1500, 600, 520), cuda)
        torch.cuda.synchronize()
        return lambda: (la.gated_ffn(q["x"], q["w"], q["w_up"], q["y"], saved=q["saved"], stream=stream),
                        la.gated_ffn_backward(q["x"], q["w"], q["w_up"], q["saved"], q["dy"], q["dx"], q["dw"], q["dw_up"],
                                              workspace=q["ws"], stream=stream))
    names = ("y", "dx", "dw", "dw_up")
    for q in (c, d):
        run(q, None)()
    want = [[q[n].clone() for n in names] for q in (c, d)]
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for q in (c, d):
        for n in names:
            q[n].zero_()
    one, two = run(c, s), run(d, t.cuda_stream)
    for _ in range(4):
        one()
        two()
    torch.cuda.synchronize()
    for q, ref in zip((c, d), want):
        assert all(torch.equal(q[n], r) for n, r in zip(names, ref))
    with torch.cuda.stream(s):  # a result made for the call belongs to the stream it runs on
        y = la.linear(c["x"], c["w"])
    z = la.linear(c["x"], c["w"], stream=s)
    s.synchronize()
    assert torch.equal(y, z)
    assert la.device_status() == 0


def test_captured_and_replayed(cuda):
    """Forward and backward pass of the block in a graph, replayed with other inputs in the same places, between
    eager calls that use the same workspace in stream order."""
    g = torch.Generator().manual_seed(8)
    m, D, F = 520, 264, 400
    weights = [(torch.randn(*s, generator=g) * sd).to(BF16).to(cuda) for s, sd in
               (((D,), 1.0), ((D,), 0.2), ((F, D), D ** -0.5), ((F, D), D ** -0.5), ((D, F), F ** -0.5))]
    block = FeedForward(m, *weights, train=True)
    x, dy = torch.empty(m, D, dtype=BF16, device=cuda), torch.empty(m, D, dtype=BF16, device=cuda)
    inputs = [[torch.randn(m, D, generator=g).to(BF16).to(cuda) for _ in range(2)] for _ in range(3)]
    keep = lambda: [block.y.clone()] + [t.clone() for t in block.grads.values()]  # noqa: E731
    want = []
    for a, b in inputs:
        x.copy_(a), dy.copy_(b)
        block.forward(x), block.backward(dy)
        want.append(keep())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.forward(x)
        block.backward(dy)
    for (a, b), ref in zip(inputs, want):
        x.copy_(a), dy.copy_(b)
        graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(keep(), ref))
        block.forward(x), block.backward(dy)
        assert all(torch.equal(p, q) for p, q in zip(keep(), ref))
    assert la.device_status() == 0


def test_the_wait_runs_out(cuda, monkeypatch):
    """A block that waits for what never comes gives up, says so, and leaves the context usable: tiles by pairs of
    blocks, and split sums."""
    c, d, f = case(cuda, 1030, 2000, 264, 9), case(cuda, 8, 400, 2000, 10), case(cuda, 777, 5001, 2048, 11)
    want = [la.linear(q["x"], q["w"]).clone() for q in (c, d, f)]
    torch.cuda.synchronize()
    assert la.device_status() == 0
    monkeypatch.setenv("LA_WAIT_LIMIT_NS", "20000000")
    for q in (c, d, f):
        monkeypatch.setenv("LA_DEBUG_STALL", "1")
        la.linear(q["x"], q["w"], q["y"])
        assert la.device_status() & 2
        monkeypatch.delenv("LA_DEBUG_STALL")
    for q, ref in zip((c, d, f), want):
        assert torch.equal(la.linear(q["x"], q["w"]), ref)
    assert la.device_status() == 0


# ---------------------------------------------------------------------------------- the whole block
def block64(x, norm_w, norm_b, w_gate, w_up, w_down, act):
    var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
    n = (x - mean) / torch.sqrt(var + 1e-5) * norm_w + norm_b
    return (act64(n @ w_gate.T, act) * (n @ w_up.T)) @ w_down.T + x


@pytest.mark.parametrize("m,D,F,act", [(1, 64, 128, "silu"), (37, 200, 333, "gelu"), (600, 1000, 1500, "silu"), (3000, 264, 700, "gelu_tanh")])
def test_feed_forward(cuda, m, D, F, act):
    """y and every gradient against the 64-bit block, and every gradient against differences of it.

    Norm-wise bounds: each of the roundings on the way (n, gate, up, h, y; dh, dgate, dup, dn, dx) moves its values by
    at most U of themselves, that is a relative U in norm, and passes on through products and norms whose gain in
    norm is at most 4 here (weights of unit gain, |act'| <= 1.13, norm weights around 1). Ten of them: 40 U, taken as
    if none cancelled."""
    g = torch.Generator().manual_seed(m + D)
    shapes = ((m, D), (D,), (D,), (F, D), (F, D), (D, F))
    scales = (1.0, 0.2, 0.2, D ** -0.5, D ** -0.5, F ** -0.5)
    t = [(torch.randn(*s, generator=g) * sd + (1.0 if i == 1 else 0.0)).to(BF16).to(cuda) for i, (s, sd) in enumerate(zip(shapes, scales))]
    t = [rows_like(v) if v.dim() == 2 else v for v in t]
    dy = rows((m, D), BF16, cuda, g)
    block = FeedForward(m, *t[1:], act=act, train=True)
    y = block.forward(t[0]).clone()
    grads = block.backward(dy)
    torch.cuda.synchronize()
    assert la.device_status() == 0
    leaves = [v.double().requires_grad_() for v in t]
    ref = block64(*leaves, act)
    want = torch.autograd.grad(ref, leaves, dy.double())
    near = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert near(y, ref.detach()) <= 40 * U
    names = ("x", "norm_w", "norm_b", "w_gate", "w_up", "w_down")
    for name, w in zip(names, want):
        assert near(grads[name], w) <= 40 * U, (name, near(grads[name], w))
    # differences: (L(p + e d) - L(p - e d)) / 2 e = <gradient, d> + O(e^2); e = 1e-4 leaves 1e-7 of third derivatives of
    # order 10 and 1e-11 of rounding in 64 bits, next to 40 U of the gradient's norm times d's
    loss = lambda *p: (block64(*p, act) * dy.double()).sum()  # noqa: E731
    with torch.no_grad():
        for i, name in enumerate(names):
            base = [v.double() for v in t]
            d = torch.randn(base[i].shape, generator=g, dtype=torch.float64).to(cuda) * base[i].abs().mean()
            up, down = [list(base) for _ in range(2)]
            up[i], down[i] = base[i] + 1e-4 * d, base[i] - 1e-4 * d
            slope = float(loss(*up) - loss(*down)) / 2e-4
            got = float((grads[name].double() * d).sum())
            assert abs(got - slope) <= 40 * U * float(want[i].norm() * d.norm()) + 1e-6 * abs(slope), name


def rows_like(v):
    out = out_rows(v.shape, v.dtype, v.device)
    out.copy_(v)
    return out


def test_feed_forward_rows_one_by_one(cuda):
    """A decode step of some streams gives what one pass over the same rows gives, to the last places of fp32 sums."""
    g = torch.Generator().manual_seed(11)
    D, F, m = 512, 1000, 300
    t = [(torch.randn(*s, generator=g) * sd).to(BF16).to(cuda) for s, sd in
         (((D,), 1.0), ((F, D), D ** -0.5), ((F, D), D ** -0.5), ((D, F), F ** -0.5))]
    x = torch.randn(m, D, generator=g).to(BF16).to(cuda)
    many = FeedForward(m, t[0], None, *t[1:]).forward(x)
    step = FeedForward(4, t[0], None, *t[1:])
    for i in range(0, m, 60):
        got = step.forward(x[i:i + 4])
        # h is rounded once in each; a sum at the edge of a step may round the other way: one step of h, U |h| |Wd| a term
        near = float((got.double() - many[i:i + 4].double()).norm() / many[i:i + 4].double().norm())
        assert near <= 4 * U


def test_feed_forward_refusals(cuda):
    w = lambda *s: torch.zeros(*s, dtype=BF16, device=cuda)  # noqa: E731
    for name, bad in (("w_down", dict(w_down=w(128, 64))), ("w_up", dict(w_up=w(128, 64).float())), ("w_gate", dict(w_gate=w(64, 128).t())),
                      ("w_gate", dict(w_gate=w(128, 67)[:, :64])), ("norm_w", dict(norm_w=w(128)[::2])), ("norm_b", dict(norm_b=w(65)[1:])),
                      ("w_up", dict(w_up=torch.zeros(128, 64, dtype=BF16)))):
        with pytest.raises(ValueError, match=name):
            FeedForward(4, **(dict(norm_w=w(64), norm_b=None, w_gate=w(128, 64), w_up=w(128, 64), w_down=w(64, 128)) | bad))
    block = FeedForward(4, w(64), None, w(128, 64), w(128, 64), w(64, 128))
    with pytest.raises(RuntimeError, match="train"):
        block.backward(w(4, 64))
    with pytest.raises(RuntimeError, match="forward"):
        FeedForward(4, w(64), None, w(128, 64), w(128, 64), w(64, 128), train=True).backward(w(4, 64))
    with pytest.raises(ValueError, match="y"):
        block.forward(w(5, 64))
    for bad in (w(4, 64).float(), w(4, 63)):
        with pytest.raises((TypeError, ValueError)):
            block.forward(bad)
    with pytest.raises(TypeError):
        la.linear(w(4, 64), w(8, 64), bias=torch.zeros(8, device=cuda))
    with pytest.raises(la.LinAttnError, match="16 bytes"):
        la.linear(w(4, 64), w(8, 64), residual=w(4, 9)[:, :8])
    with pytest.raises(la.LinAttnError, match="workspace"):
        la.linear_backward(w(4, 64), w(8, 64), None, w(4, 8), w(4, 64))
