"""The gated recurrent layer's operators together, as they are used: a training pass of conv1d + SiLU and
the scan against automatic differentiation in 64 bits, a decode loop with 4-bit projections against the
calls one by one and against the plain layer, and phase 1 with 4-bit weights."""
import numpy as np
import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la
from linear_attention_chunked_conv1d_gb300.inputs import WORKLOADS
from linear_attention_chunked_conv1d_gb300.path import GatedDecode, GatedPass, Phase1
from tests.helpers import f64

pytestmark = pytest.mark.gpu


def layer64(x, ab, conv_w, conv_bias, conv_state, h, lengths):
    """The plain layer in 64 bits, differentiable: y, the windows and the states it leaves."""
    K, C = conv_w.shape[1], x.shape[1]
    ys, windows, states, t0 = [], [], [], 0
    for s, n in enumerate(lengths):
        rows = torch.cat([conv_state[s], x[t0:t0 + n]])
        state = h[s]
        for t in range(n):
            p = conv_bias + (rows[t:t + K] * conv_w.t()).sum(0)
            u = p * torch.sigmoid(p)
            a, b = ab[t0 + t, :C], ab[t0 + t, C:]
            state = (1 - torch.sigmoid(a)) * state + torch.sigmoid(b) * u
            ys.append(state)
        windows.append(rows[n:])
        states.append(state)
        t0 += n
    return torch.stack(ys), torch.stack(windows), torch.stack(states)


def test_training_pass(cuda):
    """Every gradient, of a loss over y and the states left behind. Gates within 4 keep the memory under
    60 tokens; each of the three kernels is off by a few 2^-20 of its own operands (their own tests),
    which the sums over tokens average: 2^-15 of a gradient's largest value is a factor of ten more."""
    lengths, C, K = [70, 0, 1, 33, 130], 40, 4
    T, B = sum(lengths), len(lengths)
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    host = dict(x=r(T, C), ab=r(T, 2 * C).clamp(-4, 4), conv_w=0.5 * r(C, K), conv_bias=r(C),
                conv_state=r(B, K - 1, C), h=r(B, C))
    dy, dwindow, dstate = r(T, C), r(B, K - 1, C), r(B, C)
    v = {n: u.double().requires_grad_() for n, u in host.items()}
    y, windows, states = layer64(**v, lengths=lengths)
    ((y * dy).sum() + (windows * dwindow).sum() + (states * dstate).sum()).backward()

    inp = {n: u.to(cuda) for n, u in host.items()}
    inp["cu_seqlens"] = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=cuda)
    p = GatedPass(inp, train=True)
    for _ in range(2):  # a second step from the same states gives the same
        for n in ("conv_state", "h"):
            inp[n].copy_(host[n])
        got_y = p.forward()
        dw, ds = dwindow.to(cuda), dstate.to(cuda)
        grads = p.backward(dy.to(cuda), dh_final_ptrs=la.pointer_array(list(ds)),
                           dconv_final_ptrs=la.pointer_array(list(dw)))
        torch.cuda.synchronize()
        assert la.device_status() == 0
        for got, want in ((got_y, y), (inp["h"], states), (inp["conv_state"], windows)):
            want = want.detach().numpy()
            assert np.max(np.abs(f64(got) - want)) <= 2.0 ** -15 * np.max(np.abs(want))
        for n, got in grads.items():
            want = v[n].grad.numpy()
            assert np.max(np.abs(f64(got) - want)) <= 2.0 ** -15 * np.max(np.abs(want)), n


def test_training_pass_in_two_pieces_matches_one(cuda):
    """Truncating nothing: the gradients of the states that the second piece started from, handed to the
    first piece as those of the states it left, give the whole sequence's gradients."""
    C, K, T, cut = 24, 4, 300, 111
    g = torch.Generator().manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    host = dict(x=r(T, C), ab=r(T, 2 * C).clamp(-4, 4), conv_w=0.5 * r(C, K), conv_bias=r(C),
                conv_state=r(1, K - 1, C), h=r(1, C))
    dy = r(T, C).to(cuda)

    def a_pass(lo, hi, conv_state, h):
        inp = {n: u.to(cuda) for n, u in host.items()}
        inp.update(x=inp["x"][lo:hi], ab=inp["ab"][lo:hi], conv_state=conv_state.clone(), h=h.clone(),
                   cu_seqlens=torch.tensor([0, hi - lo], dtype=torch.int32, device=cuda))
        p = GatedPass(inp, train=True)
        p.forward()
        return p, inp

    whole, _ = a_pass(0, T, host["conv_state"].to(cuda), host["h"].to(cuda))
    want = {n: u.clone() for n, u in whole.backward(dy).items()}
    one, inp = a_pass(0, cut, host["conv_state"].to(cuda), host["h"].to(cuda))
    two, _ = a_pass(cut, T, inp["conv_state"], inp["h"])
    g2 = two.backward(dy[cut:])
    g1 = one.backward(dy[:cut], dh_final_ptrs=la.pointer_array(list(g2["h"])),
                      dconv_final_ptrs=la.pointer_array(list(g2["conv_state"])))
    torch.cuda.synchronize()
    for n in ("x", "ab"):
        got = torch.cat([g1[n], g2[n]])
        assert float((got - want[n]).abs().max()) <= 2.0 ** -15 * float(want[n].abs().max()), n
    for n in ("conv_w", "conv_bias"):
        assert float((g1[n] + g2[n] - want[n]).abs().max()) <= 2.0 ** -15 * float(want[n].abs().max()), n
    for n in ("h", "conv_state"):
        assert float((g1[n] - want[n]).abs().max()) <= 2.0 ** -15 * float(want[n].abs().max()), n


@pytest.mark.parametrize("B", [1, 5, 32])
def test_decode_loop(cuda, B):
    """Prompts through GatedPass, then tokens through GatedDecode with 4-bit projections: the states are
    the plain layer's, fed with the rows that the projection gave."""
    C, D, K, steps = 96, 256, 4, 3
    g = torch.Generator().manual_seed(3 + B)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(cuda)  # noqa: E731
    norm_w, conv_w, bias = r(D), (0.5 * r(C, K)).contiguous(), r(C)
    w_in = la.w4_quantize((r(3 * C, D) / D ** 0.5).contiguous(), group=64)
    w_out = la.w4_quantize((r(D, C) / C ** 0.5).contiguous(), group=32)
    lengths = [7 + 3 * (s % 4) for s in range(B)]
    T = sum(lengths)
    inp = dict(x=r(T, C), ab=r(T, 2 * C), conv_w=conv_w, conv_bias=bias, conv_state=r(B, K - 1, C),
               h=torch.randn(B, C, generator=g).to(cuda),
               cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=cuda))
    GatedPass(inp).forward()
    state, win = f64(inp["h"]), f64(inp["conv_state"])
    layer = GatedDecode(norm_w, w_in, w_out, conv_w, bias, inp["conv_state"], inp["h"])
    for t in range(steps):
        out = layer.run(r(B, D))
        torch.cuda.synchronize()
        x, ab = f64(layer.rows[:, :C]), f64(layer.rows[:, C:])
        xh = np.concatenate([win, x[:, None]], 1)
        p = f64(bias) + np.einsum("bkc,ck->bc", xh, f64(conv_w))
        keep, beta = 1 / (1 + np.exp(ab[:, :C])), 1 / (1 + np.exp(-ab[:, C:]))
        state, win = keep * state + beta * p / (1 + np.exp(-p)), xh[:, 1:]
        # three steps, each under 2^-19 of its operands (those of the conv: up to 10)
        assert np.max(np.abs(f64(inp["h"]) - state) / np.maximum(np.abs(state), 1.0)) <= 2.0 ** -14
        assert np.array_equal(f64(inp["conv_state"]), win)
        assert np.all(np.abs(f64(layer.y) - state) <= 2.0 ** -8 * np.abs(state) + 2.0 ** -13)
        assert out.shape == (B, D) and bool(torch.isfinite(out).all())


def test_decode_path_object(cuda):
    """GatedDecode.run against the calls one by one, for 4-bit and for bf16 weights."""
    B, C, D, K = 6, 128, 256, 3
    g = torch.Generator().manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(cuda)  # noqa: E731
    norm_w, conv_w, bias = r(D), (0.5 * r(C, K)).contiguous(), r(C)
    dense_in, dense_out = (r(3 * C, D) / D ** 0.5).contiguous(), (r(D, C) / C ** 0.5).contiguous()
    for w_in, w_out in (((la.w4_quantize(dense_in)), (la.w4_quantize(dense_out))), (dense_in, dense_out)):
        window, h = r(B, K - 1, C), torch.randn(B, C, generator=g).to(cuda)
        window2, h2 = window.clone(), h.clone()
        layer = GatedDecode(norm_w, w_in, w_out, conv_w, bias, window, h)
        for _ in range(3):
            hidden = r(B, D)
            got = layer.run(hidden).clone()
            mul = la.w4_matvec if isinstance(w_in, tuple) else (lambda v, w: la.gemm_bf16(v, w))
            args = (lambda w: w) if isinstance(w_in, tuple) else (lambda w: (w,))
            rows = mul(la.rmsnorm_rows(hidden, norm_w), *args(w_in))
            y = torch.empty(B, C, dtype=torch.bfloat16, device=cuda)
            la.gated_scan_step(la.pointer_array(list(h2)), rows[:, :C], rows[:, C:], y, conv_w=conv_w, conv_bias=bias,
                               conv_state_ptrs=la.pointer_array(list(window2)))
            want = mul(y, *args(w_out))
            torch.cuda.synchronize()
            assert torch.equal(got, want) and torch.equal(h, h2) and torch.equal(window, window2)


def test_phase1_with_4_bit_weights(cuda):
    """Phase 1 of a decode step: every output against the 64-bit products of its own stage's inputs."""
    wl = WORKLOADS["gdn_varlen_32_hk16_hv32_d128"].replace(B=4, Hk=1, Hv=2)
    D, t = 256, 4
    g = torch.Generator().manual_seed(10)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(cuda)  # noqa: E731
    dense = [(r(n, D) / D ** 0.5).contiguous() for n in (wl.cd, wl.Hv * wl.d, 2 * wl.Hv)]
    w = [la.w4_quantize(v, group=32) for v in dense]
    norm_w, hidden = r(D), r(t, D)
    out = Phase1(wl, norm_w, *w).run(hidden)
    torch.cuda.synchronize()
    assert torch.equal(out["x"], la.w4_matvec(out["y"], *w[0])) and torch.equal(out["z"], la.w4_matvec(out["y"], *w[1]))
    assert torch.equal(out["ab"], la.w4_matvec(out["y"], *w[2]))
    a, b = f64(out["ab"][:, :wl.Hv]), f64(out["ab"][:, wl.Hv:])
    assert np.max(np.abs(f64(out["g"]) + np.logaddexp(0, a))) <= 1e-5
    assert np.max(np.abs(f64(out["beta"]) - 1 / (1 + np.exp(-b)))) <= 1e-6
    assert out["x"].shape == (t, wl.cd) and out["z"].shape == (t, wl.Hv * wl.d)


def test_scan_wait_runs_out_then_next_call_is_correct(cuda, monkeypatch):
    """With LA_DEBUG_STALL=1 a tile's search of its chain finds nothing; after LA_WAIT_LIMIT_NS the call
    gives up, every block leaves, the status says so, and the next call runs."""
    T, C = 3000, 64
    g = torch.Generator().manual_seed(11)
    x, ab = torch.randn(T, C, generator=g).to(cuda), torch.randn(T, 2 * C, generator=g).to(cuda)
    ws = torch.empty(la.gated_scan_workspace_bytes(1, T, C, x.dtype), dtype=torch.uint8, device=cuda)
    saved = torch.empty(la.gated_scan_saved_bytes(1, T, C, x.dtype), dtype=torch.uint8, device=cuda)
    y, dx, dab = torch.empty_like(x), torch.empty_like(x), torch.empty_like(ab)

    def call():
        la.gated_scan(None, x, ab, y, saved=saved, workspace=ws)
        first = la.device_status()
        la.gated_scan_backward(x, ab, saved, x, dx, dab, workspace=ws)
        return first, la.device_status()

    assert call() == (0, 0)
    want = [v.clone() for v in (y, dx, dab)]
    monkeypatch.setenv("LA_DEBUG_STALL", "1")
    monkeypatch.setenv("LA_WAIT_LIMIT_NS", "1000000")
    assert call() == (la.LA_DEV_TIMEOUT, la.LA_DEV_TIMEOUT)
    monkeypatch.delenv("LA_DEBUG_STALL")
    monkeypatch.delenv("LA_WAIT_LIMIT_NS")
    assert call() == (0, 0)
    for u, v in zip((y, dx, dab), want):
        assert torch.equal(u, v)


def test_binding_refuses_what_does_not_fit(cuda):
    """Shapes, types and layouts that the calls cannot take raise before anything runs."""
    B, C, K = 3, 16, 4
    bf = dict(dtype=torch.bfloat16, device=cuda)
    x, ab, y = torch.zeros(B, C, **bf), torch.zeros(B, 2 * C, **bf), torch.full((B, C), 5.0, **bf)
    h, win = torch.zeros(B, C, device=cuda), torch.zeros(B, K - 1, C, **bf)
    hp, wp = la.pointer_array(list(h)), la.pointer_array(list(win))
    w, bias = torch.zeros(C, K, **bf), torch.zeros(C, **bf)
    step = lambda *a, **kw: la.gated_scan_step(*a, **{**dict(conv_state_ptrs=wp, conv_w=w, conv_bias=bias), **kw})  # noqa: E731
    for args, kw, kind, match in (
            ((hp, x, ab[:, :C], y), {}, ValueError, "ab"), ((hp, x, ab.float(), y), {}, TypeError, "ab"),
            ((hp, x, ab, y[:2]), {}, ValueError, "y"), ((hp[:2], x, ab, y), {}, ValueError, "h_state_ptrs"),
            ((hp, x.t().contiguous().t(), ab, y), {}, ValueError, "x"), ((hp.float(), x, ab, y), {}, TypeError, "h_state"),
            ((hp, x, ab, y), dict(conv_w=w[:8]), ValueError, "conv_w"), ((hp, x, ab, y), dict(conv_w=w.float()), TypeError, "conv_w"),
            ((hp, x, ab, y), dict(conv_bias=bias[:8]), ValueError, "conv_bias"),
            ((hp, x, ab, y), dict(conv_state_ptrs=wp[:1]), ValueError, "conv_state_ptrs"),
            ((hp, x, ab, y), dict(conv_state_ptrs=None), la.LinAttnError, "conv_state_ptrs"),
            ((None, x, ab, y), {}, la.LinAttnError, "h_state_ptrs"),
            ((hp, x, ab, y), dict(max_streams=2), la.LinAttnError, "max_streams"),
            ((hp.cpu(), x, ab, y), {}, ValueError, "h_state_ptrs"), ((hp, x, ab, x), {}, la.LinAttnError, "alias")):
        with pytest.raises(kind, match=match):
            step(*args, **kw)
    v, q, s = torch.zeros(2, 64, **bf), torch.zeros(8, 32, dtype=torch.uint8, device=cuda), torch.zeros(8, 2, **bf)
    for args, kind, match in (((v.float(), q, s), TypeError, "x"), ((v, q[:4], s), ValueError, "q"), ((v, q.int(), s), TypeError, "q"),
                              ((v, q, s[:, :0]), ValueError, "scales"), ((v, q, s, torch.zeros(2, 7, **bf)), ValueError, "y"),
                              ((v, q, s, torch.zeros(8, 2, **bf).t()), ValueError, "y"), ((v, q, s.float()), TypeError, "scales"),
                              ((torch.zeros(33, 64, **bf), q, s), la.LinAttnError, "rows")):
        with pytest.raises(kind, match=match):
            la.w4_matvec(*args)
    T = 20
    x, ab, y = torch.zeros(T, C, **bf), torch.zeros(T, 2 * C, **bf), torch.full((T, C), 5.0, **bf)
    cu = torch.tensor([0, 5, T], dtype=torch.int32, device=cuda)
    ws = torch.empty(la.gated_scan_workspace_bytes(2, T, C, x.dtype), dtype=torch.uint8, device=cuda)
    for args, kw, kind, match in (
            ((None, x, ab, y, cu.long()), {}, TypeError, "cu_seqlens"), ((None, x, ab, y, cu), dict(B=3), ValueError, "B = 3"),
            ((hp, x, ab, y, cu), {}, ValueError, "h_state_ptrs"), ((None, x, ab, y, cu), dict(workspace=None), la.LinAttnError, "workspace"),
            ((None, x, ab, y, cu), dict(workspace=ws[:8]), la.LinAttnError, "workspace"),
            ((None, x, ab, y, cu), dict(saved=ws[:8]), la.LinAttnError, "saved"), ((None, x, ab[:10], y, cu), {}, ValueError, "ab"),
            ((None, x, ab, y, None), dict(B=3), la.LinAttnError, "multiple")):
        with pytest.raises(kind, match=match):
            la.gated_scan(*args, **{**dict(workspace=ws), **kw})
    torch.cuda.synchronize()
    assert torch.all(y == 5.0) and la.device_status() == 0


@pytest.mark.parametrize("K", [1, 4])
@pytest.mark.parametrize("raw", [False, True])
def test_pass_on_a_stream_and_without_bias(cuda, K, raw):
    """GatedPass on a stream of the caller's (torch's object or its raw handle), its first kernel held back
    by work of that stream, gives what it gives on the current one; without a bias there is no gradient of it."""
    lengths, C = [70, 0, 131], 32
    T, B = sum(lengths), len(lengths)
    g = torch.Generator().manual_seed(20)
    r = lambda *s: torch.randn(*s, generator=g).to(cuda)  # noqa: E731
    inp = dict(x=r(T, C), ab=r(T, 2 * C), conv_w=0.5 * r(C, K), conv_bias=None, conv_state=r(B, K - 1, C), h=r(B, C),
               cu_seqlens=torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=cuda))
    start = inp["conv_state"].clone(), inp["h"].clone()
    dy = r(T, C)
    p = GatedPass(inp, train=True)
    want = p.forward().clone(), {n: u if u is None else u.clone() for n, u in p.backward(dy).items()}, inp["h"].clone()
    assert want[1]["conv_bias"] is None
    for n, u in zip(("conv_state", "h"), start):
        inp[n].zero_()
    p = GatedPass(inp, train=True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        busy = torch.randn(4096, 4096, device=cuda)
        for _ in range(8):
            busy = (busy @ busy).clamp(-1, 1)
        for n, u in zip(("conv_state", "h"), start):
            inp[n].copy_(u)
    stream = side.cuda_stream if raw else side
    y = p.forward(stream=stream)
    grads = p.backward(dy, stream=stream)
    side.synchronize()
    assert la.device_status(side) == 0
    assert torch.equal(y, want[0]) and torch.equal(inp["h"], want[2])
    for n, u in grads.items():
        assert (u is None and want[1][n] is None) or torch.equal(u, want[1][n]), n
    with pytest.raises(RuntimeError, match="train"):
        GatedPass(inp).backward(dy)


@pytest.mark.parametrize("raw", [False, True])
def test_products_allocate_on_the_stream_they_run_on(cuda, raw):
    """A result that is allocated for a side stream does not take memory that work of the current stream
    may still write to: the block that the current stream has just freed is not the result's."""
    N, K = 512, 256
    g = torch.Generator().manual_seed(21)
    w = torch.randn(N, K, generator=g).to(torch.bfloat16).to(cuda)
    x = torch.randn(4, K, generator=g).to(torch.bfloat16).to(cuda)
    want_q, want_s = la.w4_quantize(w)
    want = la.w4_matvec(x, want_q, want_s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream = side.cuda_stream if raw else side
    freed = [torch.empty(n, dtype=torch.uint8, device=cuda) for n in (N * K // 2, N * K // 128 * 2, 4 * N * 2)]
    places = {u.data_ptr() for u in freed}
    del freed
    q, s = la.w4_quantize(w, stream=stream)
    y = la.w4_matvec(x, q, s, stream=stream)
    side.synchronize()
    assert not places & {q.data_ptr(), s.data_ptr(), y.data_ptr()}
    assert torch.equal(q, want_q) and torch.equal(s, want_s) and torch.equal(y, want)


def test_a_single_row_may_come_from_a_matrix_of_any_width(cuda):
    """One token of a wider matrix whose row stride is no multiple of 16 bytes: the stride says nothing."""
    C, wide = 64, 259
    g = torch.Generator().manual_seed(22)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(cuda)  # noqa: E731
    x, ab, dy = r(3, wide)[:1, :C], r(3, wide)[:1, :2 * C], r(3, wide)[:1, :C]
    w = r(C, 4)
    outs = []
    for f in (lambda v: v, lambda v: v.contiguous()):
        y, dx, dab = torch.empty_like(x), torch.empty(1, C, device=cuda, dtype=x.dtype), torch.empty(1, 2 * C, device=cuda, dtype=x.dtype)
        ws = torch.empty(la.gated_scan_workspace_bytes(1, 1, C, x.dtype), dtype=torch.uint8, device=cuda)
        saved = torch.empty(la.gated_scan_saved_bytes(1, 1, C, x.dtype), dtype=torch.uint8, device=cuda)
        la.gated_scan(None, f(x), f(ab), y, saved=saved, workspace=ws)
        la.gated_scan_backward(f(x), f(ab), saved, f(dy), dx, dab, workspace=ws)
        dw, dcx = torch.empty(C, 4, device=cuda), torch.empty_like(dx)
        cws = torch.empty(la.conv1d_silu_backward_workspace_bytes(1, 1, C, 4, x.dtype), dtype=torch.uint8, device=cuda)
        window = torch.zeros(1, 3, C, device=cuda, dtype=x.dtype)
        la.conv1d_silu_backward(la.pointer_array(list(window)), f(x), w, f(dy), dcx, dw, workspace=cws)
        q, s = la.w4_quantize(r(3, wide)[:1, :C] * 0 + 1, group=32)
        outs.append((y, dx, dab, dcx, dw, la.w4_matvec(f(x), q, s)))
    torch.cuda.synchronize()
    assert la.device_status() == 0
    for u, v in zip(*outs):
        assert torch.equal(u, v)
    with pytest.raises(ValueError, match="groups of 0"):
        la.w4_quantize(w, group=0)


def test_calls_next_to_copies_fills_and_another_stream(cuda):
    """Launches overlap the end of the kernel before them, and wait for it: whatever stands before a call in
    its stream (a copy, a fill, another call, the event of another stream), it reads what that wrote and
    writes only then. Eager and in a captured graph, many times over, bit for bit as with a wait of the host
    after every call."""
    C, K, T, lengths = 256, 4, 700, [300, 0, 400]
    g = torch.Generator().manual_seed(23)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(cuda)  # noqa: E731
    x0, ab0, dy0, w, rows0 = r(T, C), r(T, 2 * C), r(T, C), r(C, K), r(3, C)
    qs = [la.w4_quantize((r(n, C) / 16).contiguous(), group=64) for n in (3 * C, C)]
    h0, win0 = torch.randn(3, C, generator=g).to(cuda), r(3, K - 1, C)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device=cuda)
    x, ab, dy, rows = (torch.empty_like(v) for v in (x0, ab0, dy0, rows0))
    h, win = torch.empty_like(h0), torch.empty_like(win0)
    hp, wp = la.pointer_array(list(h)), la.pointer_array(list(win))
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=cuda)  # noqa: E731
    y, dx, dab, dcx, dw = e(T, C), e(T, C), e(T, 2 * C), e(T, C), e(C, K, dtype=torch.float32)
    step, tri, back = e(3, C), e(3, 3 * C), e(3, C)
    ws, ws2 = e(la.gated_scan_workspace_bytes(3, T, C, x.dtype), dtype=torch.uint8), e(1 << 20, dtype=torch.uint8)
    saved = e(la.gated_scan_saved_bytes(3, T, C, x.dtype), dtype=torch.uint8)
    assert la.conv1d_silu_backward_workspace_bytes(3, T, C, K, x.dtype) <= ws2.numel()
    total = torch.zeros((), device=cuda)
    side = torch.cuda.Stream()

    def work(wait):
        main = torch.cuda.current_stream()
        for a, b in ((x, x0), (ab, ab0), (dy, dy0), (h, h0), (win, win0)):
            a.copy_(b)
        wait()
        la.gated_scan(hp, x, ab, y, cu, saved=saved, workspace=ws)
        wait()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            rows.copy_(rows0)
            la.w4_matvec(rows, *qs[0], tri)
            wait()
            la.gated_scan_step(hp, tri[:, :C], tri[:, C:], step, conv_state_ptrs=wp, conv_w=w)
            wait()
            la.w4_matvec(step, *qs[1], back)
            wait()
            back.mul_(2)
        x.zero_()  # the scan has read it; the backward pass gets it back
        x.copy_(x0)
        la.gated_scan_backward(x, ab, saved, dy, dx, dab, cu, workspace=ws)
        wait()
        main.wait_stream(side)
        la.conv1d_silu_backward(wp, x, w, dx, dcx, dw, cu, workspace=ws2)
        wait()
        dx.add_(back[0])
        la.w4_matvec(dx[:3], *qs[1], step)
        total.add_(step.float().sum() + dcx.float().sum() + dw.sum())

    outs = (y, dx, dab, dcx, dw, step, tri, back, h, win)
    work(torch.cuda.synchronize)
    torch.cuda.synchronize()
    want = [v.clone() for v in outs]
    assert all(bool(torch.isfinite(v).all()) for v in want)
    for v in outs:
        v.zero_()
    for _ in range(20):
        work(lambda: None)
    torch.cuda.synchronize()
    for u, v in zip(outs, want):
        assert torch.equal(u, v)
        u.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(lambda: None)
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert la.device_status() == 0
    for u, v in zip(outs, want):
        assert torch.equal(u, v)


def test_handle_zero_is_the_default_stream(cuda):
    """stream=0 from within another stream: the pass's copy of the windows and its kernels come after what the
    default stream holds, and what the products allocate is that stream's."""
    T, C, K = 50, 32, 4
    g = torch.Generator().manual_seed(24)
    r = lambda *s: torch.randn(*s, generator=g).to(cuda)  # noqa: E731
    start = r(1, K - 1, C)
    inp = dict(x=r(T, C), ab=r(T, 2 * C), conv_w=r(C, K), conv_bias=None, conv_state=torch.zeros_like(start),
               h=torch.zeros(1, C, device=cuda), cu_seqlens=torch.tensor([0, T], dtype=torch.int32, device=cuda))
    p = GatedPass(inp, train=True)
    w = la.w4_quantize(torch.randn(256, 256, generator=g).to(torch.bfloat16).to(cuda))
    x4 = torch.randn(4, 256, generator=g).to(torch.bfloat16).to(cuda)
    want = la.w4_matvec(x4, *w)
    busy = r(4096, 4096)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    for _ in range(8):
        busy = (busy @ busy).clamp(-1, 1)
    inp["conv_state"].copy_(start)
    freed = torch.empty(4 * 256 * 2, dtype=torch.uint8, device=cuda)
    place = freed.data_ptr()
    del freed
    with torch.cuda.stream(side):
        p.forward(stream=0)
        y = la.w4_matvec(x4, *w, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(p.conv_start, start) and y.data_ptr() == place and torch.equal(y, want)
