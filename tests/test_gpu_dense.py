"""The dense half of a layer against plain forms in 64 bits: layer norm, products with bias, activation
and residual, the gated feed-forward block, and their backward passes.

Bounds. u = torch.finfo(bf16).eps / 2 = 2^-8 is half a step of bf16 relative to the value (7 stored fraction
bits: steps of 2^-7 between 1 and 2; fp32: 2^-24); a result rounded once is off
by u |ref|. Sums of n terms in fp32 add at most n 2^-24 sum |terms|, in practice far less: 64 2^-24 sum |terms|
covers the split sums used here. Where an operand of a product was itself rounded to bf16 (dz, dgate, dup
from values kept in bf16), every term may be off by what its factor is:
  z, gate, up kept in bf16: u each, times the sensitivity of act' (|z act''| <= 1.2 for every activation here,
  act <= |z|), then u for the rounding of dz: at most 4 u of dy (1 + |z|) |up| a term; the bound below takes the
  sums of absolute terms, as no cancellation is assumed.
"""
import math

import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la

pytestmark = pytest.mark.gpu

U, F32 = torch.finfo(torch.bfloat16).eps / 2, torch.finfo(torch.float32).eps / 2
ACTS = list(la.LA_ACTIVATIONS)


def rows(shape, dtype, cuda, g, std=1.0, extra=0):
    """A matrix with rows on 16 bytes and NaN in what lies between them."""
    per = 16 // dtype.itemsize
    ld = (shape[1] + per - 1) // per * per + extra
    t = torch.full((shape[0], ld), float("nan"), dtype=dtype)
    t[:, :shape[1]] = torch.randn(shape, generator=g) * std
    return t.to(cuda)[:, :shape[1]]


def out_rows(shape, dtype, cuda, extra=0):
    per = 16 // dtype.itemsize
    ld = (shape[1] + per - 1) // per * per + extra
    return torch.full((shape[0], ld), 7.0, dtype=dtype, device=cuda)[:, :shape[1]]


def untouched(t):
    """What lies between the rows of a matrix of out_rows."""
    full = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1))
    return bool((full[:, t.shape[1]:] == 7.0).all())


def act64(z, act):
    return {"none": lambda: z, "relu": lambda: torch.clamp_min(z, 0), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: 0.5 * z * torch.erfc(-z / math.sqrt(2)),
            # (1 + tanh u) / 2 = 1 / (1 + e^-2u), which keeps the left tail that 1 + tanh u loses in 64 bits too
            "gelu_tanh": lambda: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))}[act]()


def slope64(z, act):
    z = z.detach().requires_grad_()
    with torch.enable_grad():
        return torch.autograd.grad(act64(z, act).sum(), z)[0]


def close(got, ref, bound, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (what, int(bad.sum()), float(err[bad].max()), float((err / bound)[bad].max()))


# ---------------------------------------------------------------------------------- layer norm
NORMS = [(1, 1), (1, 8), (3, 7), (5, 64), (9, 250), (33, 256), (17, 257), (40, 512), (700, 513), (2, 1000), (1300, 1024), (31, 2047),
         (700, 2048), (12, 4096), (5, 4099), (650, 5000), (3, 8191), (7, 8192)]


def norm_bound(dt):
    return U if dt == torch.bfloat16 else 8 * F32


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m,n", NORMS)
def test_layernorm(cuda, m, n, dt):
    g = torch.Generator().manual_seed(m * 10007 + n)
    x, dy, dskip = (rows((m, n), dt, cuda, g, extra=16 * i) for i in range(3))
    x += torch.randn(m, 1, generator=g).to(cuda).to(dt)
    w = (1 + 0.3 * torch.randn(n, generator=g)).to(dt).to(cuda)
    b = torch.randn(n, generator=g).to(dt).to(cuda)
    y, dx = out_rows((m, n), dt, cuda, 8), out_rows((m, n), dt, cuda)
    stats = torch.full((m, 2), 7.0, device=cuda)
    dw, db = torch.full((n,), 7.0, device=cuda), torch.full((n,), 7.0, device=cuda)
    ws = torch.full((la.layernorm_rows_backward_workspace_bytes(m, n, dt),), 255, dtype=torch.uint8, device=cuda)
    eps = 1e-5
    assert la.layernorm_rows(x, w, b, y, stats=stats, eps=eps) is y
    la.layernorm_rows_backward(x, w, stats, dy, dx, dw, db, dskip=dskip, workspace=ws)
    torch.cuda.synchronize()

    X, W, B, DY = x.double(), w.double(), b.double(), dy.double()
    mean = X.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((X - mean) ** 2).mean(1, keepdim=True) + eps)
    xh = (X - mean) * rstd
    # what fp32 statistics add: the mean's and variance's sums, relative to the row's largest value
    big = X.abs().amax(1, keepdim=True) * rstd
    stat = 64 * F32 * (big + xh.abs() + 1)
    assert (stats[:, :1].double() - mean).abs().max() <= 16 * F32 * X.abs().amax()
    close(stats[:, 1:], rstd, 64 * F32 * rstd * (1 + big ** 2 / max(n, 1)), "rstd")
    # rstd's error grows where a row is flat against its mean (width 1: the variance is 0)
    ref = xh * W + B
    close(y, ref, norm_bound(dt) * ref.abs() + stat * W.abs() + 4 * F32 * B.abs(), "y")
    u = DY * W
    ref = rstd * (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True)) + dskip.double()
    size = rstd * (u.abs() + u.abs().mean(1, keepdim=True) + (xh.abs() + stat) * (u * xh).abs().mean(1, keepdim=True)
                   + xh.abs() * u.abs().mean(1, keepdim=True) * stat.amax(1, keepdim=True) * 1e3)
    close(dx, ref, norm_bound(dt) * ref.abs() + 64 * F32 * size * (1 + big) + 4 * F32 * dskip.double().abs(), "dx")
    close(dw, (DY * xh).sum(0), (DY.abs() * (stat + 64 * F32 * xh.abs())).sum(0), "dw")
    close(db, DY.sum(0), 64 * F32 * DY.abs().sum(0), "db")
    assert untouched(y) and untouched(dx)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_layernorm_in_place_without_bias_and_skip(cuda, dt):
    g = torch.Generator().manual_seed(5)
    m, n = 300, 1000
    x, dy, dskip = (rows((m, n), dt, cuda, g) for _ in range(3))
    w = (1 + 0.3 * torch.randn(n, generator=g)).to(dt).to(cuda)
    stats = torch.empty(m, 2, device=cuda)
    y = la.layernorm_rows(x, w, stats=stats)
    xi = x.clone(memory_format=torch.preserve_format)
    la.layernorm_rows(xi, w, y=xi)
    assert torch.equal(xi, y)
    ws = torch.empty(la.layernorm_rows_backward_workspace_bytes(m, n, dt), dtype=torch.uint8, device=cuda)
    grads = []
    for how in range(4):
        skip = dskip.clone() if how in (1, 3) else None
        d = dy.clone()
        dx = torch.empty_like(d) if how < 2 else d if how == 2 else skip
        dw = torch.empty(n, device=cuda)
        la.layernorm_rows_backward(x, w, stats, d, dx, dw, dskip=skip, workspace=ws)
        grads.append((dx, dw))
    torch.cuda.synchronize()
    assert torch.equal(grads[0][0], grads[2][0]) and torch.equal(grads[1][0], grads[3][0])
    assert all(torch.equal(grads[0][1], gw) for _, gw in grads)


def test_layernorm_rows_do_not_touch_one_another(cuda):
    """A row of NaN, one of infinities and one without any spread leave the others as they are."""
    g = torch.Generator().manual_seed(6)
    for n in (100, 3000):
        x = rows((64, n), torch.bfloat16, cuda, g)
        w = torch.ones(n, dtype=torch.bfloat16, device=cuda)
        good = la.layernorm_rows(x, w).clone()
        x[3], x[17, 5], x[40] = float("nan"), float("inf"), 2.5
        got = la.layernorm_rows(x, w)
        keep = [r for r in range(64) if r not in (3, 17, 40)]
        assert torch.equal(got[keep], good[keep])
        assert got[3].isnan().all() and got[17].isnan().all() and (got[40] == 0).all()


# ---------------------------------------------------------------------------------- products
SHAPES = [(1, 1, 1), (1, 8, 8), (2, 3, 5), (1, 300, 129), (7, 1001, 264), (33, 130, 1000), (64, 64, 64), (100, 129, 72), (129, 257, 130),
          (255, 64, 63), (300, 520, 200), (513, 1025, 513), (1000, 333, 2049)]


def case(cuda, m, n, k, seed, bias=True, residual=True):
    g = torch.Generator().manual_seed(seed)
    bf16 = torch.bfloat16
    return dict(x=rows((m, k), bf16, cuda, g, extra=8), w=rows((n, k), bf16, cuda, g, 1 / math.sqrt(k)),
                bias=torch.randn(n, generator=g).to(bf16).to(cuda) if bias else None,
                residual=rows((m, n), bf16, cuda, g, extra=16) if residual else None,
                dy=rows((m, n), bf16, cuda, g, extra=24), y=out_rows((m, n), bf16, cuda),
                dx=out_rows((m, k), bf16, cuda, 8), dw=out_rows((n, k), bf16, cuda, 16),
                dbias=torch.full((n,), 7.0, dtype=bf16, device=cuda))


def room(n, cuda):
    return torch.full((n,), 255, dtype=torch.uint8, device=cuda)


def check_linear(c, act, backward=True):
    """One forward and backward call, against 64 bits."""
    cuda, (m, k), n = c["x"].device, c["x"].shape, c["w"].shape[0]
    X, W, DY = c["x"].double(), c["w"].double(), c["dy"].double()
    saved = room(la.linear_saved_bytes(m, n, act), cuda) if backward else None
    assert la.linear(c["x"], c["w"], c["y"], bias=c["bias"], residual=c["residual"], act=act, saved=saved) is c["y"]
    if backward:
        la.linear_backward(c["x"], c["w"], saved, c["dy"], c["dx"], c["dw"], dbias=c["dbias"], act=act,
                           workspace=room(la.linear_backward_workspace_bytes(m, n, k, act), cuda))
    torch.cuda.synchronize()
    assert la.device_status() == 0
    Bi = c["bias"].double() if c["bias"] is not None else torch.zeros(n, device=cuda, dtype=torch.float64)
    R = c["residual"].double() if c["residual"] is not None else torch.zeros(m, n, device=cuda, dtype=torch.float64)
    z = X @ W.T + Bi
    mag = X.abs() @ W.abs().T + Bi.abs()
    ref = act64(z, act) + R
    close(c["y"], ref, U * ref.abs() + 64 * F32 * (1.2 * mag + ref.abs() + R.abs()), "y")
    assert untouched(c["y"])
    if not backward:
        return
    dz = DY * slope64(z, act)
    per = (0 if act == "none" else 4 * U) * DY.abs() * (1 + z.abs()) + 64 * F32 * DY.abs() * (1 + mag)
    if act == "relu":  # a z within the sums' error of 0 may fall on either side of the step
        per = torch.where(dz == 0, 0.0, U * dz.abs()) + torch.where(z.abs() <= 64 * F32 * mag, DY.abs(), 0.0)
    for name, got, ref, bound in (("dx", c["dx"], dz @ W, (per + 64 * F32 * dz.abs()) @ W.abs()),
                                  ("dw", c["dw"], dz.T @ X, (per + 64 * F32 * dz.abs()).T @ X.abs()),
                                  ("dbias", c["dbias"], dz.sum(0), (per + 64 * F32 * dz.abs()).sum(0))):
        close(got, ref, U * ref.abs() + bound + 1e-30, name)
    assert untouched(c["dx"]) and untouched(c["dw"])


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(cuda, m, n, k):
    for i, act in enumerate(ACTS):
        check_linear(case(cuda, m, n, k, 100 * m + n + k, bias=i % 2 == 0, residual=i % 3 != 1), act)


# ---------------------------------------------------------------------------------- gated block
def check_gated(c, act, backward=True):
    cuda, (m, k), f = c["x"].device, c["x"].shape, c["w"].shape[0]
    X, G, Uw, DH = c["x"].double(), c["w"].double(), c["w_up"].double(), c["dy"].double()
    saved = room(la.gated_ffn_saved_bytes(m, f), cuda) if backward else None
    assert la.gated_ffn(c["x"], c["w"], c["w_up"], c["y"], act=act, saved=saved) is c["y"]
    if backward:
        la.gated_ffn_backward(c["x"], c["w"], c["w_up"], saved, c["dy"], c["dx"], c["dw"], c["dw_up"], act=act,
                              workspace=room(la.gated_ffn_backward_workspace_bytes(m, f, k), cuda))
    torch.cuda.synchronize()
    assert la.device_status() == 0
    gate, up = X @ G.T, X @ Uw.T
    mg, mu = X.abs() @ G.abs().T, X.abs() @ Uw.abs().T
    a = act64(gate, act)
    ref = a * up
    close(c["y"], ref, U * ref.abs() + 64 * F32 * (1.2 * mg * up.abs() + a.abs() * mu + 1.2 * F32 * 64 * mg * mu + ref.abs()), "h")
    assert untouched(c["y"])
    if not backward:
        return
    dg, du = DH * up * slope64(gate, act), DH * a
    per_g = DH.abs() * (5 * U * up.abs() * (1 + gate.abs()) + 64 * F32 * (mu * (1 + gate.abs()) + up.abs() * (1 + mg)))
    per_u = DH.abs() * (3 * U * (1.2 * gate.abs() + a.abs()) + 64 * F32 * (1 + mg))
    if act == "relu":
        per_g += torch.where(gate.abs() <= 64 * F32 * mg, (DH * up).abs(), 0.0)
    close(c["dx"], dg @ G + du @ Uw, U * (dg @ G + du @ Uw).abs() + (per_g + 64 * F32 * dg.abs()) @ G.abs()
          + (per_u + 64 * F32 * du.abs()) @ Uw.abs(), "dx")
    close(c["dw"], dg.T @ X, U * (dg.T @ X).abs() + (per_g + 64 * F32 * dg.abs()).T @ X.abs(), "dw_gate")
    close(c["dw_up"], du.T @ X, U * (du.T @ X).abs() + (per_u + 64 * F32 * du.abs()).T @ X.abs(), "dw_up")
    assert untouched(c["dx"]) and untouched(c["dw"]) and untouched(c["dw_up"])


def gated_case(cuda, m, f, k, seed):
    c = case(cuda, m, f, k, seed, bias=False, residual=False)
    g = torch.Generator().manual_seed(seed + 1)
    c["w_up"] = rows((f, k), torch.bfloat16, cuda, g, 1 / math.sqrt(k), extra=8)
    c["dw_up"] = out_rows((f, k), torch.bfloat16, cuda)
    return c


@pytest.mark.parametrize("m,f,k", SHAPES)
def test_gated_ffn(cuda, m, f, k):
    for act in ACTS:
        check_gated(gated_case(cuda, m, f, k, 7 * m + f + k), act)
