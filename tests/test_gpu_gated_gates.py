"""The gated recurrence (scan, backward pass, decode step) with gates anywhere from -80 to 80: decays,
input gates and the complements of both to their own last places, so that a gradient through a gate that is
nearly open or shut is right relative to itself.

Bounds. Of a gate v the smaller side is 2^-|t| / (1 + 2^-|t|), t = |v| log2 e: the constant's and the product's
roundings move it by 1.5 |v| 2^-24 relative to it, the hardware exponential and reciprocal by 2^-22 + 2^-23,
three roundings by 3 * 2^-24: E(v) = |v| 2^-23 + 2^-21 together. The larger side is off by the smaller one's
error and one rounding. A token adds those for its two gates and four roundings (joins of runs among them) of
what it keeps and takes, k |h| and beta |x|; all of it decays with k. Results below 1e-37 are not looked at."""
import numpy as np
import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la
from tests.helpers import f64
from tests.test_gpu_gated_scan import DT, close, gpu_pass, make

pytestmark = pytest.mark.gpu

ROUND = 2.0 ** -22


def sides(v):
    """sigmoid(v), sigmoid(-v) and the bounds of their errors."""
    up, down = 1 / (1 + np.exp(-v)), 1 / (1 + np.exp(v))
    e = np.minimum(up, down) * (abs(v) * 2.0 ** -23 + 2.0 ** -21)
    return up, down, e + 2.0 ** -24 * up, e + 2.0 ** -24 * down


def reference(x, ab, h0, dy, dfinal, lengths):
    C = x.shape[1]
    d, keep, d_e, keep_e = sides(ab[:, :C])
    beta, rest, beta_e, rest_e = sides(ab[:, C:])
    z = lambda: np.zeros_like(x)  # noqa: E731
    y, y_e, before, before_e, lam, lam_e = z(), z(), z(), z(), z(), z()
    fin, fin_e, dh0, dh0_e = h0.copy(), 0 * h0, dfinal.copy(), 0 * h0
    t0 = 0
    for s, n in enumerate(lengths):
        h, e = h0[s].copy(), np.zeros(C)
        for t in range(t0, t0 + n):
            before[t], before_e[t] = h, e
            u = beta[t] * x[t]
            e = keep[t] * e + keep_e[t] * abs(h) + beta_e[t] * abs(x[t]) + ROUND * (keep[t] * abs(h) + abs(u))
            h = keep[t] * h + u
            y[t], y_e[t] = h, e
        fin[s], fin_e[s] = h, e
        m, e = dfinal[s].copy(), np.zeros(C)
        for t in range(t0 + n - 1, t0 - 1, -1):
            lam[t], lam_e[t] = dy[t] + m, e + ROUND * (abs(dy[t]) + abs(m))
            e = keep[t] * lam_e[t] + (keep_e[t] + ROUND * keep[t]) * abs(lam[t])
            m = keep[t] * lam[t]
        dh0[s], dh0_e[s] = m, e
        t0 += n
    dx, db, da = lam * beta, lam * x * beta * rest, -lam * before * d * keep
    dx_e = lam_e * beta + abs(lam) * beta_e + 2.0 ** -24 * abs(dx)
    gate = lambda p, q, p_e, q_e: p_e * q + p * q_e + 2.0 ** -22 * p * q  # noqa: E731
    db_e = lam_e * abs(x) * beta * rest + abs(lam * x) * gate(beta, rest, beta_e, rest_e)
    da_e = (lam_e * abs(before) + abs(lam) * before_e) * d * keep + abs(lam * before) * gate(d, keep, d_e, keep_e)
    return dict(y=(y, y_e), h=(fin, fin_e), dx=(dx, dx_e), dab=(np.concatenate([da, db], 1), np.concatenate([da_e, db_e], 1)),
                dh0=(dh0, dh0_e))


def check(cuda, inp, lengths, dtype):
    want = reference(*(f64(inp[n]) for n in ("x", "ab", "h", "dy", "dfinal")), lengths)
    for (name, (v, e)), got in zip(want.items(), gpu_pass(cuda, inp, lengths)):
        close(got, v, e, "f32" if name in ("h", "dh0") else dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[1] * 40, [100], [700], [64, 300, 0, 256, 37]], ids=["ones", "one tile", "chain", "packed"])
@pytest.mark.parametrize("most", [12.0, 30.0, 80.0])
def test_gates_of_any_size(cuda, most, lengths, dtype):
    """Both gates uniform over -most .. most."""
    inp = make(lengths, 72, dtype, seed=70)
    g = torch.Generator().manual_seed(int(most))
    inp["ab"] = (most * (2 * torch.rand(inp["ab"].shape, generator=g) - 1)).to(DT[dtype])
    check(cuda, inp, lengths, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_gate_for_each_channel(cuda, dtype):
    """Channels with the same gates at every token: a from -20 to 20 (with +-0), b the other way."""
    lengths, C = [700, 40], 72
    inp = make(lengths, C, dtype, seed=71)
    a = torch.linspace(-20, 20, C)
    a[7], a[8] = 0.0, -0.0
    inp["ab"] = torch.cat([a, -a]).expand(sum(lengths), 2 * C).to(DT[dtype]).contiguous()
    check(cuda, inp, lengths, dtype)


def test_a_channel_that_forgets_less_than_a_rounding(cuda):
    """a = -17: d = 4.1e-8 is under one step of 1 - d, and 20,000 tokens lose 8.2e-4 of a state. A tile's decay is
    applied as h - d h with one rounding (2^-25): 79 tiles forward and 157 backward stay under 4.7e-6; y has, in
    its tile, at most 16 more in its run and 62 in the joins of runs, 2.4e-6."""
    T, C = 20000, 8
    inp = dict(x=torch.zeros(T, C), ab=torch.full((T, 2 * C), -17.0), h=torch.ones(1, C), dy=torch.zeros(T, C), dfinal=torch.ones(1, C))
    y, h, dx, dab, dh0 = gpu_pass(cuda, inp, [T])
    d = 1 / (1 + np.exp(17.0))
    want = np.exp(np.arange(1, T + 1) * np.log1p(-d))
    assert np.max(abs(f64(y)[:, 0] / want - 1)) <= 4.7e-6 + 2.4e-6
    assert np.max(abs(f64(h) / want[-1] - 1)) <= 4.7e-6 and np.max(abs(f64(dh0) / want[-1] - 1)) <= 4.7e-6


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gradients_of_infinite_gates(cuda, dtype):
    """Gates of +-infinity pass no gradient to themselves, whole or none of it to x, and all or nothing back."""
    inf, (T, C) = float("inf"), (300, 32)
    inp = make([T], C, dtype, seed=72)
    ab = inp["ab"].float()
    ab[:, 0:8], ab[:, C:C + 8] = -inf, inf          # h += x
    ab[:, 8:16], ab[:, C + 8:C + 16] = inf, inf     # h = x
    ab[:, 16:24], ab[:, C + 16:C + 24] = -inf, -inf  # h stays
    inp["ab"] = ab.to(DT[dtype])
    inp["x"], inp["dy"] = torch.randint(-3, 4, (T, C)).to(DT[dtype]), torch.randint(-3, 4, (T, C)).to(DT[dtype])
    inp["h"], inp["dfinal"] = torch.ones(1, C), torch.full((1, C), 2.0)
    y, h, dx, dab, dh0 = (f64(v) for v in gpu_pass(cuda, inp, [T]))
    x, dy = f64(inp["x"]), f64(inp["dy"])
    back = np.cumsum(dy[::-1], 0)[::-1] + 2.0  # whole numbers under 2^11: exact in fp32, one rounding in bf16
    near = lambda u, v: np.all(abs(u - v) <= abs(v) * (2.0 ** -8 if dtype == "bf16" else 0.0))  # noqa: E731
    assert np.array_equal(h[0, :8], 1 + x[:, :8].sum(0)) and np.array_equal(h[0, 8:16], x[-1, 8:16]) and np.all(h[0, 16:24] == 1)
    assert near(dx[:, :8], back[:, :8]) and np.array_equal(dx[:-1, 8:16], dy[:-1, 8:16]) and np.all(dx[:, 16:24] == 0)
    assert np.array_equal(dh0[0, :8], back[0, :8]) and np.all(dh0[0, 8:16] == 0) and np.array_equal(dh0[0, 16:24], back[0, 16:24])
    assert np.all(abs(dab[:, :24]) < 1e-37) and np.all(abs(dab[:, C:C + 24]) < 1e-37)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_with_gates_of_any_size(cuda, dtype):
    B, C = 40, 72
    inp = make([B], C, dtype, seed=73)
    g = torch.Generator().manual_seed(74)
    ab = (80 * (2 * torch.rand(B, 2 * C, generator=g) - 1)).to(DT[dtype])
    h = 1e4 * torch.randn(B, C, generator=g)
    want = reference(f64(inp["x"]), f64(ab), f64(h), 0 * f64(inp["x"]), 0 * f64(h), [1] * B)
    hd, y = h.clone().to(cuda), torch.empty(B, C, dtype=DT[dtype], device=cuda)
    la.gated_scan_step(la.pointer_array(list(hd)), inp["x"].to(cuda), ab.to(cuda), y)
    torch.cuda.synchronize()
    close(hd, *want["h"])
    close(y, *want["y"], dtype)
